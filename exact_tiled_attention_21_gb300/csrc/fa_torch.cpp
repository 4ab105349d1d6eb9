// Native binding of the serving-cache conveniences (rope, cache_append_fp8,
// decode_paged_fp8, cache_evict_fp8): checks the tensors, allocates the outputs
// and the workspace with torch on its current stream, and calls the C ABI.  The
// same steps in Python took 21 to 40 us of host time per call, these take 4 to
// 10; the small calls take about 4 us on the GPU.
//
// Each function takes its arguments by position, from the Python function of the
// same name, and returns its result, or the status of a C call that failed.
#include <Python.h>

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

#define FA_FN(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_FN(rope), FA_FN(append), FA_FN(decode), FA_FN(evict), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module); }
