// Native binding of the serving-cache conveniences (rope, cache_append_fp8,
// decode_paged_fp8, cache_evict_fp8 and, for the bf16 cache, cache_append,
// select_blocks, decode_blocks, decode_shared): checks the tensors, allocates the outputs
// and the workspace with torch on its current stream, and calls the C ABI.  The
// same steps in Python took 21 to 40 us of host time per call, these take 4 to
// 10; the small calls take about 4 us on the GPU.
//
// Each function takes its arguments by position, from the Python function of the
// same name, and returns its result, or the status of a C call that failed.
#include <Python.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fa.h"

namespace {

using at::Tensor;

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// A contiguous tensor of this type, shape and device; its pointer.
void* checked(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
    const Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.device() == dev && t.sizes() == shape && t.is_contiguous(), name,
                      " must be a contiguous ", type, " tensor of shape ", shape, " on ", dev);
    return t.data_ptr();
}

void* optional(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
    return o == Py_None ? nullptr : checked(o, name, type, shape, dev);
}

// Counts a write in place, so that autograd refuses a gradient that would take the old values.
void written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();  // inference tensors have no counter
}
void written(PyObject* o) { written(THPVariable_Unpack(o)); }

// A bf16 CUDA tensor [B, H, N, d] whose innermost dimension is dense.
const Tensor& bhnd(PyObject* o, const char* name) {
    const Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == at::kBFloat16 && t.dim() == 4, name,
                      " must be a bf16 CUDA tensor [B, H, N, d]");
    TORCH_CHECK_VALUE(t.stride(3) == 1, name, " must be dense in its last dimension");
    return t;
}

int size(int64_t n, const char* name) {
    TORCH_CHECK_VALUE(n <= INT_MAX, name, " is too large");
    return (int)n;
}

Tensor make(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// The turns table: its pointer and the number of rotated columns.
const uint64_t* turns_of(PyObject* o, c10::Device dev, int* rot) {
    const Tensor& t = tensor(o, "turns");
    TORCH_CHECK_VALUE(t.dim() == 1, "turns must have one dimension");
    *rot = size(2 * t.size(0), "turns");
    return static_cast<const uint64_t*>(checked(o, "turns", at::kLong, t.sizes(), dev));
}

struct Cache {
    c10::Device dev = c10::Device(c10::kCPU);
    int B, Hkv, page, d, sb, max_pages, num_pages;
    void *k, *v, *ks, *vs, *table, *lens;

    explicit Cache(PyObject* const* o) {
        const Tensor &kp = tensor(o[0], "k_pages"), &sc = tensor(o[2], "k_scale"), &tab = tensor(o[4], "block_table");
        TORCH_CHECK_VALUE(kp.is_cuda() && kp.dim() == 4, "k_pages must be a CUDA tensor [num_pages, Hkv, page, d]");
        TORCH_CHECK_VALUE(sc.dim() == 3 && sc.size(0) == kp.size(0) && sc.size(1) == kp.size(1) && sc.size(2) >= 1 &&
                              kp.size(2) % sc.size(2) == 0,
                          "k_scale must have shape [num_pages, Hkv, a divisor of the page size]");
        TORCH_CHECK_VALUE(tab.dim() == 2, "block_table must have 2 dimensions");
        dev = kp.device();
        k = checked(o[0], "k_pages", at::kByte, kp.sizes(), dev);
        v = checked(o[1], "v_pages", at::kByte, kp.sizes(), dev);
        ks = checked(o[2], "k_scale", at::kFloat, sc.sizes(), dev);
        vs = checked(o[3], "v_scale", at::kFloat, sc.sizes(), dev);
        table = checked(o[4], "block_table", at::kInt, tab.sizes(), dev);
        lens = checked(o[5], "seq_lens", at::kInt, {tab.size(0)}, dev);
        num_pages = size(kp.size(0), "num_pages");
        Hkv = size(kp.size(1), "Hkv");
        page = size(kp.size(2), "page");
        d = size(kp.size(3), "d");
        sb = (int)(page / sc.size(2));
        B = size(tab.size(0), "B");
        max_pages = size(tab.size(1), "max_pages");
    }
    int64_t tokens() const { return (int64_t)max_pages * page; }
};

// Runs a C call without the GIL.
template <typename F>
int call(F f) {
    int st;
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS return st;
}

PyObject* status(int st) { return PyLong_FromLong(st); }

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return false;
}

float number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)x;
}

int integer(PyObject* o) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(x >= INT_MIN && x <= INT_MAX, "integer out of range");
    return (int)x;
}

int truth(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x;
}

// rope(x, turns, positions, interleaved, magnitude, inverse, out)
PyObject* rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (!count(n, 7)) return nullptr;
    HANDLE_TH_ERRORS
    const Tensor& x = bhnd(o[0], "x");
    const c10::Device dev = x.device();
    int rot;
    const uint64_t* turns = turns_of(o[1], dev, &rot);
    const auto pos = static_cast<const int*>(optional(o[2], "positions", at::kInt, {x.size(0), x.size(2)}, dev));
    const int inter = truth(o[3]), inverse = truth(o[5]);
    const float magnitude = number(o[4]);
    const c10::cuda::CUDAGuard guard(dev);
    Tensor y;
    if (o[6] == Py_None) {
        y = make(x.sizes(), at::kBFloat16, dev);
    } else {
        y = bhnd(o[6], "out");
        TORCH_CHECK_VALUE(y.sizes() == x.sizes() && y.device() == dev, "out must have x's shape and device");
    }
    const int B = size(x.size(0), "B"), H = size(x.size(1), "H"), N = size(x.size(2), "N"), d = size(x.size(3), "d");
    void* stream = stream_of(dev);
    const int st = call([&] {
        return fa_rope(x.data_ptr(), y.data_ptr(), x.stride(0), x.stride(1), x.stride(2), y.stride(0), y.stride(1),
                       y.stride(2), pos, turns, B, H, N, d, rot, inter, magnitude, inverse, stream);
    });
    if (st != FA_OK) return status(st);
    if (o[6] != Py_None) written(y);
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

// cache_append_fp8(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, new_lens, turns, positions,
//                  interleaved, magnitude)
PyObject* append(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (!count(n, 13)) return nullptr;
    HANDLE_TH_ERRORS
    const Cache c(o + 2);
    const Tensor &k = bhnd(o[0], "k"), &v = bhnd(o[1], "v");
    TORCH_CHECK_VALUE(k.device() == c.dev && v.device() == c.dev && k.size(0) == c.B && k.size(1) == c.Hkv &&
                          k.size(3) == c.d && v.sizes() == k.sizes(),
                      "k and v must have shape [B, Hkv, N, d], on the cache's device");
    const int N = size(k.size(2), "N");
    const auto fresh = static_cast<const int*>(optional(o[8], "new_lens", at::kInt, {c.B}, c.dev));
    int rot = 0;
    const uint64_t* turns = o[9] == Py_None ? nullptr : turns_of(o[9], c.dev, &rot);
    const auto pos = static_cast<const int*>(turns ? optional(o[10], "positions", at::kInt, {c.B, N}, c.dev) : nullptr);
    const int inter = truth(o[11]);
    const float magnitude = number(o[12]);
    const c10::cuda::CUDAGuard guard(c.dev);
    void* stream = stream_of(c.dev);
    const int st = call([&] {
        return fa_cache_append_fp8(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), v.stride(0),
                                   v.stride(1), v.stride(2), c.k, c.v, (float*)c.ks, (float*)c.vs, (const int*)c.table,
                                   (const int*)c.lens, fresh, pos, turns, c.B, c.Hkv, N, c.d, rot, inter, magnitude,
                                   c.page, c.sb, c.max_pages, c.num_pages, stream);
    });
    if (st == FA_OK)
        for (int i = 2; i < 6; ++i) written(o[i]);
    return status(st);
    END_HANDLE_TH_ERRORS
}

// decode_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, scale, weights, workspace)
PyObject* decode(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (!count(n, 10)) return nullptr;
    HANDLE_TH_ERRORS
    const Cache c(o + 1);
    const Tensor& q = tensor(o[0], "q");
    const int64_t dims = q.dim();
    TORCH_CHECK_VALUE((dims == 3 || dims == 4) && q.scalar_type() == at::kBFloat16 && q.device() == c.dev &&
                          q.is_contiguous() && q.size(0) == c.B && q.size(dims - 1) == c.d,
                      "q must be a contiguous bf16 tensor [B, Hq, Nq, d] or [B, Hq, d] on the cache's device");
    const int Hq = size(q.size(1), "Hq"), Nq = dims == 4 ? size(q.size(2), "Nq") : 1;
    const float scale = o[7] == Py_None ? (float)(1.0 / std::sqrt((double)c.d)) : number(o[7]);
    const auto weights = static_cast<float*>(optional(o[8], "weights", at::kFloat, {c.B, c.Hkv, c.tokens()}, c.dev));
    const c10::cuda::CUDAGuard guard(c.dev);
    Tensor ws;
    if (o[9] == Py_None) {
        const int64_t tokens = c.tokens();
        ws = make({(int64_t)fa_decode_paged_fp8_workspace_bytes(c.B, Hq, c.Hkv, Nq, c.d, tokens <= INT_MAX ? (int)tokens : 0,
                                                                weights != nullptr)},
                  at::kByte, c.dev);
    } else {
        ws = tensor(o[9], "workspace");
        TORCH_CHECK_VALUE(ws.device() == c.dev && ws.is_contiguous(), "workspace must be contiguous, on the cache's device");
    }
    const Tensor out = make(q.sizes(), at::kBFloat16, c.dev);
    const Tensor lse = make(q.sizes().slice(0, dims - 1), at::kFloat, c.dev);
    void* stream = stream_of(c.dev);
    const int st = call([&] {
        return fa_decode_paged_fp8(q.data_ptr(), c.k, c.v, (const float*)c.ks, (const float*)c.vs, (const int*)c.table,
                                   (const int*)c.lens, out.data_ptr(), (float*)lse.data_ptr(), weights, c.B, Hq, c.Hkv, Nq,
                                   c.page, c.sb, c.max_pages, c.num_pages, c.d, scale, ws.data_ptr(), ws.nbytes(), stream);
    });
    if (st != FA_OK) return status(st);
    if (weights) written(o[8]);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
    END_HANDLE_TH_ERRORS
}

// cache_evict_fp8(k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, weights, new_table, keep, recent)
PyObject* evict(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (!count(n, 10)) return nullptr;
    HANDLE_TH_ERRORS
    const Cache c(o);
    const auto weights = static_cast<const float*>(checked(o[6], "weights", at::kFloat, {c.B, c.Hkv, c.tokens()}, c.dev));
    const Tensor& nt = tensor(o[7], "new_table");
    TORCH_CHECK_VALUE(nt.dim() == 2, "new_table must have 2 dimensions");
    const auto table = static_cast<const int*>(checked(o[7], "new_table", at::kInt, {c.B, nt.size(1)}, c.dev));
    const int new_max_pages = size(nt.size(1), "new_max_pages"), keep = integer(o[8]), recent = integer(o[9]);
    const c10::cuda::CUDAGuard guard(c.dev);
    const int64_t tokens = (int64_t)new_max_pages * c.page;
    const Tensor lens = make({c.B}, at::kInt, c.dev), w = make({c.B, c.Hkv, tokens}, at::kFloat, c.dev),
                 kept = make({c.B, c.Hkv, tokens}, at::kInt, c.dev);
    void* stream = stream_of(c.dev);
    const int st = call([&] {
        return fa_cache_evict_fp8(c.k, c.v, (float*)c.ks, (float*)c.vs, (const int*)c.table, (const int*)c.lens, weights,
                                  table, (int*)lens.data_ptr(), (float*)w.data_ptr(), (int*)kept.data_ptr(), c.B, c.Hkv,
                                  c.page, c.sb, c.max_pages, new_max_pages, c.num_pages, c.d, keep, recent, stream);
    });
    if (st != FA_OK) return status(st);
    for (int i = 0; i < 4; ++i) written(o[i]);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(lens), THPVariable_Wrap(w), THPVariable_Wrap(kept));
    END_HANDLE_TH_ERRORS
}

// The paged bf16 cache: pages, table and lengths.
struct Pages {
    c10::Device dev = c10::Device(c10::kCPU);
    int B, Hkv, page, d, max_pages, num_pages;
    void *k, *v, *table, *lens;

    Pages(PyObject* kp, PyObject* vp, PyObject* tab, PyObject* len) {
        const Tensor &p = tensor(kp, "k_pages"), &t = tensor(tab, "block_table");
        TORCH_CHECK_VALUE(p.is_cuda() && p.dim() == 4, "k_pages must be a CUDA tensor [num_pages, Hkv, page, d]");
        TORCH_CHECK_VALUE(t.dim() == 2, "block_table must have 2 dimensions");
        dev = p.device();
        k = checked(kp, "k_pages", at::kBFloat16, p.sizes(), dev);
        v = checked(vp, "v_pages", at::kBFloat16, p.sizes(), dev);
        table = checked(tab, "block_table", at::kInt, t.sizes(), dev);
        lens = checked(len, "seq_lens", at::kInt, {t.size(0)}, dev);
        num_pages = size(p.size(0), "num_pages");
        Hkv = size(p.size(1), "Hkv");
        page = size(p.size(2), "page");
        d = size(p.size(3), "d");
        B = size(t.size(0), "B");
        max_pages = size(t.size(1), "max_pages");
    }
};

// q [B, Hq, Nq, d], or [B, Hq, d] for one new token.
struct Queries {
    const Tensor& t;
    int Hq, Nq;

    Queries(PyObject* o, c10::Device dev, int B, int d) : t(tensor(o, "q")) {
        const int64_t dims = t.dim();
        TORCH_CHECK_VALUE((dims == 3 || dims == 4) && t.scalar_type() == at::kBFloat16 && t.device() == dev &&
                              t.is_contiguous() && t.size(0) == B && t.size(dims - 1) == d,
                          "q must be a contiguous bf16 tensor [B, Hq, Nq, d] or [B, Hq, d] on the cache's device");
        Hq = size(t.size(1), "Hq");
        Nq = dims == 4 ? size(t.size(2), "Nq") : 1;
    }
};

Tensor workspace(PyObject* o, size_t bytes, c10::Device dev) {
    if (o == Py_None) return make({(int64_t)bytes}, at::kByte, dev);
    const Tensor& t = tensor(o, "workspace");
    TORCH_CHECK_VALUE(t.device() == dev && t.is_contiguous(), "workspace must be contiguous, on the cache's device");
    return t;
}

// cache_append(k, v, k_pages, v_pages, block_table, seq_lens, new_lens, turns, positions, interleaved, magnitude, bounds)
PyObject* paged_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (!count(n, 12)) return nullptr;
    HANDLE_TH_ERRORS
    const Pages c(o[2], o[3], o[4], o[5]);
    const Tensor &k = bhnd(o[0], "k"), &v = bhnd(o[1], "v");
    TORCH_CHECK_VALUE(k.device() == c.dev && v.device() == c.dev && k.size(0) == c.B && k.size(1) == c.Hkv &&
                          k.size(3) == c.d && v.sizes() == k.sizes(),
                      "k and v must have shape [B, Hkv, N, d], on the cache's device");
    const int N = size(k.size(2), "N");
    const auto fresh = static_cast<const int*>(optional(o[6], "new_lens", at::kInt, {c.B}, c.dev));
    int rot = 0, block = 1;
    const uint64_t* turns = o[7] == Py_None ? nullptr : turns_of(o[7], c.dev, &rot);
    const auto pos = static_cast<const int*>(turns ? optional(o[8], "positions", at::kInt, {c.B, N}, c.dev) : nullptr);
    const int inter = truth(o[9]);
    const float magnitude = number(o[10]);
    void* bounds = nullptr;
    if (o[11] != Py_None) {
        const Tensor& t = tensor(o[11], "bounds");
        TORCH_CHECK_VALUE(t.dim() == 5 && t.size(2) >= 1 && c.page % t.size(2) == 0,
                          "bounds must have shape [num_pages, Hkv, a divisor of the page size, 2, d]");
        bounds = checked(o[11], "bounds", at::kBFloat16, {c.num_pages, c.Hkv, t.size(2), 2, c.d}, c.dev);
        block = (int)(c.page / t.size(2));
    }
    const c10::cuda::CUDAGuard guard(c.dev);
    void* stream = stream_of(c.dev);
    const int st = call([&] {
        return fa_cache_append(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), v.stride(0), v.stride(1),
                               v.stride(2), c.k, c.v, bounds, (const int*)c.table, (const int*)c.lens, fresh, pos, turns,
                               c.B, c.Hkv, N, c.d, rot, inter, magnitude, c.page, block, c.max_pages, c.num_pages, stream);
    });
    if (st == FA_OK) {
        written(o[2]);
        written(o[3]);
        if (bounds) written(o[11]);
    }
    return status(st);
    END_HANDLE_TH_ERRORS
}

// select_blocks(q, bounds, block_table, seq_lens, block, keep, first, recent, workspace)
PyObject* select_blocks(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (!count(n, 9)) return nullptr;
    HANDLE_TH_ERRORS
    const Tensor &bounds = tensor(o[1], "bounds"), &tab = tensor(o[2], "block_table");
    TORCH_CHECK_VALUE(bounds.is_cuda() && bounds.dim() == 5 && bounds.size(3) == 2,
                      "bounds must be a CUDA tensor [num_pages, Hkv, page / block, 2, d]");
    TORCH_CHECK_VALUE(tab.dim() == 2, "block_table must have 2 dimensions");
    const c10::Device dev = bounds.device();
    const void* bp = checked(o[1], "bounds", at::kBFloat16, bounds.sizes(), dev);
    const auto table = static_cast<const int*>(checked(o[2], "block_table", at::kInt, tab.sizes(), dev));
    const auto lens = static_cast<const int*>(checked(o[3], "seq_lens", at::kInt, {tab.size(0)}, dev));
    const int num_pages = size(bounds.size(0), "num_pages"), Hkv = size(bounds.size(1), "Hkv"),
              per_page = size(bounds.size(2), "page / block"), d = size(bounds.size(4), "d"), B = size(tab.size(0), "B"),
              max_pages = size(tab.size(1), "max_pages");
    const Queries q(o[0], dev, B, d);
    const int block = integer(o[4]), keep = integer(o[5]), first = integer(o[6]), recent = integer(o[7]);
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t most = (int64_t)max_pages * per_page;
    void* stream = stream_of(dev);
    auto select = [&](int* out, void* ws, size_t bytes) {
        return call([&] {
            return fa_select_blocks(q.t.data_ptr(), bp, table, lens, out, B, q.Hq, Hkv, q.Nq, block, per_page, max_pages,
                                    num_pages, d, keep, first, recent, ws, bytes, stream);
        });
    };
    if (keep > most) {  // lists longer than the table's blocks: whatever else is wrong is refused before they take memory
        const int st = select(const_cast<int*>(table), nullptr, 0);
        if (st != FA_ERR_WORKSPACE) return status(st);
    }
    const Tensor ws = workspace(o[8], fa_select_blocks_workspace_bytes(B, Hkv, most <= INT_MAX ? (int)most : 0), dev);
    const Tensor out = make({B, Hkv, std::max(keep, 0)}, at::kInt, dev);
    const int st = select((int*)out.data_ptr(), ws.data_ptr(), ws.nbytes());
    return st != FA_OK ? status(st) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// decode_blocks(q, k_pages, v_pages, block_table, seq_lens, blocks, block, scale, workspace)
PyObject* decode_blocks(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (!count(n, 9)) return nullptr;
    HANDLE_TH_ERRORS
    const Pages c(o[1], o[2], o[3], o[4]);
    const Queries q(o[0], c.dev, c.B, c.d);
    const Tensor& list = tensor(o[5], "blocks");
    TORCH_CHECK_VALUE(list.dim() == 3, "blocks must have shape [B, Hkv, keep]");
    const auto blocks = static_cast<const int*>(checked(o[5], "blocks", at::kInt, {c.B, c.Hkv, list.size(2)}, c.dev));
    const int keep = size(list.size(2), "keep"), block = integer(o[6]);
    const float scale = o[7] == Py_None ? (float)(1.0 / std::sqrt((double)c.d)) : number(o[7]);
    const c10::cuda::CUDAGuard guard(c.dev);
    const Tensor ws = workspace(o[8], fa_decode_blocks_workspace_bytes(c.B, q.Hq, c.Hkv, q.Nq, c.d), c.dev);
    const Tensor out = make(q.t.sizes(), at::kBFloat16, c.dev);
    const Tensor lse = make(q.t.sizes().slice(0, q.t.dim() - 1), at::kFloat, c.dev);
    void* stream = stream_of(c.dev);
    const int st = call([&] {
        return fa_decode_blocks(q.t.data_ptr(), c.k, c.v, (const int*)c.table, (const int*)c.lens, blocks, out.data_ptr(),
                                (float*)lse.data_ptr(), c.B, q.Hq, c.Hkv, q.Nq, c.page, block, keep, c.max_pages,
                                c.num_pages, c.d, scale, ws.data_ptr(), ws.nbytes(), stream);
    });
    if (st != FA_OK) return status(st);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
    END_HANDLE_TH_ERRORS
}

// decode_shared(q, k_pages, v_pages, block_table, seq_lens, shared_len, scale, workspace)
PyObject* decode_shared(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (!count(n, 8)) return nullptr;
    HANDLE_TH_ERRORS
    const Pages c(o[1], o[2], o[3], o[4]);
    const Queries q(o[0], c.dev, c.B, c.d);
    const auto shared = static_cast<const int*>(checked(o[5], "shared_len", at::kInt, {1}, c.dev));
    const float scale = o[6] == Py_None ? (float)(1.0 / std::sqrt((double)c.d)) : number(o[6]);
    const c10::cuda::CUDAGuard guard(c.dev);
    const Tensor ws = workspace(o[7], fa_decode_shared_workspace_bytes(c.B, q.Hq, c.Hkv, q.Nq, c.d), c.dev);
    const Tensor out = make(q.t.sizes(), at::kBFloat16, c.dev);
    const Tensor lse = make(q.t.sizes().slice(0, q.t.dim() - 1), at::kFloat, c.dev);
    void* stream = stream_of(c.dev);
    const int st = call([&] {
        return fa_decode_shared(q.t.data_ptr(), c.k, c.v, (const int*)c.table, (const int*)c.lens, shared, out.data_ptr(),
                                (float*)lse.data_ptr(), c.B, q.Hq, c.Hkv, q.Nq, c.page, c.max_pages, c.num_pages, c.d,
                                scale, ws.data_ptr(), ws.nbytes(), stream);
    });
    if (st != FA_OK) return status(st);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
    END_HANDLE_TH_ERRORS
}

#define FA_FN(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_FN(rope), FA_FN(append), FA_FN(decode), FA_FN(evict), FA_FN(paged_append),
                         FA_FN(select_blocks), FA_FN(decode_blocks), FA_FN(decode_shared), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module); }
