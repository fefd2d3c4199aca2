// bind.cpp - Python binding of the paged caches' entry points: checks tensors,
// allocates outputs and scratch, and calls the C ABI of include/attn.h on the
// current stream of the tensors' device.
//
// These calls are made at every step of a generation and often on little data,
// where the host's time counts: the same checks and allocations by ctypes and
// Python cost 10 to 14 us a call, more than most of the kernels behind them.
//
// Each function returns its result, or the C call's status (an int) where that
// is not ATTN_OK; tensors that do not fit raise ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <limits>

#include "attn.h"

namespace {

using at::Tensor;

const Tensor &tensor(PyObject *o, const char *name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// None: an undefined tensor.
const Tensor &maybe(PyObject *o, const char *name)
{
    static const Tensor none;
    return o == Py_None ? none : tensor(o, name);
}

int as_int(int64_t x, const char *name)
{
    TORCH_CHECK_VALUE(x >= 0 && x <= std::numeric_limits<int>::max(), name, " is out of range");
    return static_cast<int>(x);
}

int long_arg(PyObject *o, const char *name)
{
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(!overflow && x >= std::numeric_limits<int>::min() && x <= std::numeric_limits<int>::max(), name,
                      " is out of range");
    return static_cast<int>(x);
}

// A contiguous int32 tensor of that shape on the pages' device.
int *ints(const Tensor &t, const char *name, c10::Device device, at::IntArrayRef shape)
{
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.device() == device && t.sizes() == shape && t.is_contiguous(),
                      name, " must be a contiguous int32 tensor ", shape, " on the pages' device");
    return t.data_ptr<int>();
}

// Strides of all dimensions but the last, null if t is contiguous. A dimension
// of one element is never stepped along: its stride is given as `at_least`.
struct Strides {
    int64_t s[3];
    const int64_t *ptr = nullptr;

    void of(const Tensor &t, int64_t at_least)
    {
        if (t.is_contiguous()) return;
        const int n = static_cast<int>(t.dim()) - 1;
        // (a pool without a head dimension has one head)
        for (int i = 0; i < 3; ++i) s[i] = at_least;
        for (int i = 0; i < n; ++i)
            if (t.size(i) > 1) s[n == 2 && i == 1 ? 2 : i] = t.stride(i);
        ptr = s;
    }
};

struct Pools {
    c10::Device device;
    int heads, pages, page_size, d;
    Strides strides;
    void *k, *v = nullptr;

    Pools(const Tensor &kp, const Tensor &vp) : device(kp.device())
    {
        one(kp, "k_pages");
        if (vp.defined()) {
            one(vp, "v_pages");
            TORCH_CHECK_VALUE(kp.dim() == 4 && kp.sizes() == vp.sizes() && vp.device() == device,
                              "k_pages and v_pages must be [num_pages, Hkv, page_size, d], alike and on one device");
            v = vp.data_ptr();
        } else {
            TORCH_CHECK_VALUE(kp.dim() == 3 || kp.dim() == 4, "a single pool must be [num_pages, page_size, d] or "
                                                              "[num_pages, Hkv, page_size, d]");
        }
        k = kp.data_ptr();
        pages = as_int(kp.size(0), "num_pages");
        heads = kp.dim() == 4 ? as_int(kp.size(1), "Hkv") : 1;
        page_size = as_int(kp.size(-2), "page_size");
        d = as_int(kp.size(-1), "d");
        strides.of(kp, d);
        if (v) {
            Strides other;
            other.of(vp, d);
            bool same = (strides.ptr == nullptr) == (other.ptr == nullptr);
            for (int i = 0; same && strides.ptr && i < 3; ++i) same = strides.s[i] == other.s[i];
            TORCH_CHECK_VALUE(same, "k_pages and v_pages must have the same strides");
        }
    }

    static void one(const Tensor &t, const char *name)
    {
        TORCH_CHECK_VALUE(t.scalar_type() == at::kBFloat16 && t.is_cuda(), name, " must be a bf16 CUDA tensor");
        TORCH_CHECK_VALUE(t.dim() > 0 && (t.stride(-1) == 1 || t.size(-1) == 1), name,
                          " must be contiguous along its last dimension");
    }
};

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, c10::Device device)
{
    return at::detail::empty_cuda(shape, type, device, c10::nullopt);
}

// The caller's tensor, which has to fit, or a new one.
Tensor output(const Tensor &given, const char *name, at::IntArrayRef shape, at::ScalarType type, c10::Device device)
{
    if (!given.defined()) return fresh(shape, type, device);
    TORCH_CHECK_VALUE(given.sizes() == shape && given.scalar_type() == type && given.is_contiguous() &&
                          given.device() == device,
                      name, " must be a contiguous tensor ", shape, " of ", type, " on q's device");
    return given;
}

struct Scratch {
    Tensor t;
    void *ptr;
    size_t bytes;

    Scratch(const Tensor &given, int64_t need, const char *what, c10::Device device)
    {
        if (given.defined()) {
            TORCH_CHECK_VALUE(given.device() == device && given.is_contiguous(),
                              "workspace must be a contiguous tensor on the pages' device");
            t = given;
        } else {
            TORCH_CHECK_VALUE(need >= 0, "unsupported or invalid shape for ", what);
            t = fresh({need}, at::kByte, device);
        }
        ptr = t.data_ptr();
        bytes = t.nbytes();
    }
};

void *stream_of(c10::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

// Queries [B, H, T, d] or [B, H, d], and the tables.
struct Queries {
    int B, H, T, width;
    const int *table, *lens;

    Queries(const Tensor &q, const Pools &p, const Tensor &page_table, const Tensor &len)
    {
        TORCH_CHECK_VALUE(q.scalar_type() == at::kBFloat16 && q.device() == p.device && q.is_contiguous(),
                          "q must be a contiguous bf16 tensor on the pages' device");
        TORCH_CHECK_VALUE((q.dim() == 3 || q.dim() == 4) && q.size(-1) == p.d,
                          "q must be [B, H, T, x] or [B, H, x] with x the length of the pages' rows");
        B = as_int(q.size(0), "B");
        H = as_int(q.size(1), "H");
        T = q.dim() == 4 ? as_int(q.size(2), "T") : 1;
        TORCH_CHECK_VALUE(page_table.dim() == 2, "page_table must be [B, max_pages]");
        width = as_int(page_table.size(1), "max_pages");
        table = ints(page_table, "page_table", p.device, {B, width});
        lens = ints(len, "lens", p.device, {B});
    }
};

PyObject *pair(Tensor a, Tensor b)
{
    PyObject *x = THPVariable_Wrap(std::move(a)), *y = THPVariable_Wrap(std::move(b));
    PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

PyObject *status(int rc) { return PyLong_FromLong(rc); }

bool count_args(Py_ssize_t have, Py_ssize_t want)
{
    if (have == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
    return false;
}

// decode_paged(q, k_pages, v_pages, page_table, lens, window, scale, out, lse, workspace)
PyObject *decode_paged(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_args(n, 10)) return nullptr;
    const Tensor &q = tensor(a[0], "q");
    const Tensor &vp = tensor(a[2], "v_pages");
    const Pools p(tensor(a[1], "k_pages"), vp);
    const Queries s(q, p, tensor(a[3], "page_table"), tensor(a[4], "lens"));
    // (a window of 2^30 reaches every position there can be)
    int overflow = 0;
    long long window = PyLong_AsLongLongAndOverflow(a[5], &overflow);
    if (window == -1 && PyErr_Occurred()) throw python_error();
    window = overflow > 0 || window > (1 << 30) ? 1 << 30 : overflow < 0 || window < 0 ? -1 : window;
    const double scale = a[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(p.d)) : PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    const c10::cuda::CUDAGuard guard(p.device);
    Tensor out = output(maybe(a[7], "out"), "out", q.sizes(), at::kBFloat16, p.device);
    Tensor lse = output(maybe(a[8], "lse"), "lse", q.sizes().slice(0, q.dim() - 1), at::kFloat, p.device);
    const Tensor &given = maybe(a[9], "workspace");
    const Scratch w(given, given.defined() ? 0 : attn_decode_paged_workspace_bytes(s.B, s.H, p.heads, s.T, s.width,
                                                                                   p.page_size, p.d),
                    "attn_decode_paged", p.device);
    const int rc = attn_decode_paged(q.data_ptr(), p.k, p.v, p.strides.ptr, s.table, s.lens, out.data_ptr(),
                                     lse.data_ptr<float>(), w.ptr, w.bytes, s.B, s.H, p.heads, s.T, p.pages,
                                     p.page_size, s.width, static_cast<int>(window), p.d, static_cast<float>(scale),
                                     stream_of(p.device));
    return rc == ATTN_OK ? pair(std::move(out), std::move(lse)) : status(rc);
    END_HANDLE_TH_ERRORS
}

// decode_latent(q, pages, page_table, lens, scale, out, lse, workspace)
PyObject *decode_latent(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_args(n, 8)) return nullptr;
    const Tensor &q = tensor(a[0], "q");
    const Pools p(tensor(a[1], "pages"), Tensor());
    TORCH_CHECK_VALUE(p.heads == 1 && p.d > 64, "pages must be [num_pages, page_size, rank + 64]");
    const Queries s(q, p, tensor(a[2], "page_table"), tensor(a[3], "lens"));
    const double scale = PyFloat_AsDouble(a[4]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    const int rank = p.d - 64;
    const c10::cuda::CUDAGuard guard(p.device);
    c10::SmallVector<int64_t, 4> shape(q.sizes().begin(), q.sizes().end());
    shape.back() = rank;
    Tensor out = output(maybe(a[5], "out"), "out", shape, at::kBFloat16, p.device);
    Tensor lse = output(maybe(a[6], "lse"), "lse", q.sizes().slice(0, q.dim() - 1), at::kFloat, p.device);
    const Tensor &given = maybe(a[7], "workspace");
    const Scratch w(given, given.defined() ? 0 : attn_decode_latent_workspace_bytes(s.B, s.H, s.T, s.width,
                                                                                    p.page_size, rank),
                    "attn_decode_latent", p.device);
    const int64_t strides[2] = {p.strides.s[0], p.strides.s[2]};
    const int rc = attn_decode_latent(q.data_ptr(), p.k, p.strides.ptr ? strides : nullptr, s.table, s.lens,
                                      out.data_ptr(), lse.data_ptr<float>(), w.ptr, w.bytes, s.B, s.H, s.T, p.pages,
                                      p.page_size, s.width, rank, static_cast<float>(scale), stream_of(p.device));
    return rc == ATTN_OK ? pair(std::move(out), std::move(lse)) : status(rc);
    END_HANDLE_TH_ERRORS
}

// pages_append(k, v, k_pages, v_pages, page_table, pos, count)
PyObject *pages_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_args(n, 7)) return nullptr;
    const Tensor &k = tensor(a[0], "k"), &v = maybe(a[1], "v"), &vp = maybe(a[3], "v_pages");
    TORCH_CHECK_VALUE(v.defined() == vp.defined(), "v and v_pages go together");
    const Pools p(tensor(a[2], "k_pages"), vp);
    for (const Tensor *t : {&k, &v}) {
        if (!t->defined()) continue;
        TORCH_CHECK_VALUE(t->scalar_type() == at::kBFloat16 && t->device() == p.device && t->dim() == 4 &&
                              t->sizes() == k.sizes() && t->size(1) == p.heads && t->size(3) == p.d &&
                              t->stride(3) == 1,
                          "k and v must be bf16 tensors [B, Hkv, T, d] on the pages' device, last stride 1");
    }
    const int B = as_int(k.size(0), "B"), T = as_int(k.size(2), "T");
    const Tensor &page_table = tensor(a[4], "page_table"), &count = maybe(a[6], "count");
    TORCH_CHECK_VALUE(page_table.dim() == 2, "page_table must be [B, max_pages]");
    const int width = as_int(page_table.size(1), "max_pages");
    const int *table = ints(page_table, "page_table", p.device, {B, width});
    const int *pos = ints(tensor(a[5], "pos"), "pos", p.device, {B});
    const int *counts = count.defined() ? ints(count, "count", p.device, {B}) : nullptr;
    Strides ks, vs;
    ks.of(k, 0);
    if (v.defined()) vs.of(v, 0);
    const c10::cuda::CUDAGuard guard(p.device);
    const int rc = attn_pages_append(k.data_ptr(), v.defined() ? v.data_ptr() : nullptr, ks.ptr, vs.ptr, p.k, p.v,
                                     p.strides.ptr, table, pos, counts, B, p.heads, T, p.pages, p.page_size, width,
                                     p.d, stream_of(p.device));
    if (rc != ATTN_OK) return status(rc);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// A table and its counts.
struct State {
    c10::Device device;
    int rows, width, pages;
    int *table, *refs;

    State(const Tensor &page_table, const Tensor &counts) : device(counts.device())
    {
        TORCH_CHECK_VALUE(page_table.dim() == 2 && counts.dim() == 1 && counts.is_cuda(),
                          "page_table must be [num_rows, max_pages] and refs a CUDA tensor [num_pages]");
        rows = as_int(page_table.size(0), "num_rows");
        width = as_int(page_table.size(1), "max_pages");
        pages = as_int(counts.size(0), "num_pages");
        table = ints(page_table, "page_table", device, {rows, width});
        refs = ints(counts, "refs", device, {pages});
    }
};

// pages_reserve(page_table, refs, rows, want, page_size, workspace)
PyObject *pages_reserve(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_args(n, 6)) return nullptr;
    const State s(tensor(a[0], "page_table"), tensor(a[1], "refs"));
    const Tensor &rows = tensor(a[2], "rows");
    const int count = as_int(rows.numel(), "the number of rows");
    const int *r = ints(rows, "rows", s.device, {count});
    const int *want = ints(tensor(a[3], "want"), "want", s.device, {count});
    const int page_size = long_arg(a[4], "page_size");
    const c10::cuda::CUDAGuard guard(s.device);
    Tensor granted = fresh({count}, at::kInt, s.device);
    if (count == 0) return THPVariable_Wrap(std::move(granted));
    const Tensor &given = maybe(a[5], "workspace");
    const Scratch w(given, given.defined() ? 0 : attn_pages_workspace_bytes(count, s.rows, s.pages),
                    "the page operations", s.device);
    const int rc = attn_pages_reserve(s.table, s.refs, r, want, granted.data_ptr<int>(), w.ptr, w.bytes, count, s.rows,
                                      s.pages, page_size, s.width, stream_of(s.device));
    return rc == ATTN_OK ? THPVariable_Wrap(std::move(granted)) : status(rc);
    END_HANDLE_TH_ERRORS
}

// pages_fork(k_pages, v_pages, page_table, lens, refs, parents, children, workspace)
PyObject *pages_fork(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_args(n, 8)) return nullptr;
    const Pools p(tensor(a[0], "k_pages"), maybe(a[1], "v_pages"));
    const State s(tensor(a[2], "page_table"), tensor(a[4], "refs"));
    TORCH_CHECK_VALUE(s.device == p.device && s.pages == p.pages,
                      "refs must have one count a page, on the pages' device");
    int *const lens = ints(tensor(a[3], "lens"), "lens", p.device, {s.rows});
    const Tensor &parents = tensor(a[5], "parents");
    const int count = as_int(parents.numel(), "the number of forks");
    const int *from = ints(parents, "parents", p.device, {count});
    const int *to = ints(tensor(a[6], "children"), "children", p.device, {count});
    const c10::cuda::CUDAGuard guard(p.device);
    Tensor page = fresh({count}, at::kInt, p.device), granted = fresh({count}, at::kInt, p.device);
    if (count == 0) return pair(std::move(page), std::move(granted));
    const Tensor &given = maybe(a[7], "workspace");
    const Scratch w(given, given.defined() ? 0 : attn_pages_workspace_bytes(count, s.rows, s.pages),
                    "the page operations", p.device);
    const int rc = attn_pages_fork(p.k, p.v, p.strides.ptr, s.table, lens, s.refs, from, to, page.data_ptr<int>(),
                                   granted.data_ptr<int>(), w.ptr, w.bytes, count, s.rows, p.heads, p.pages,
                                   p.page_size, s.width, p.d, stream_of(p.device));
    return rc == ATTN_OK ? pair(std::move(page), std::move(granted)) : status(rc);
    END_HANDLE_TH_ERRORS
}

// pages_free(page_table, lens, refs, rows)
PyObject *pages_free(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_args(n, 4)) return nullptr;
    const State s(tensor(a[0], "page_table"), tensor(a[2], "refs"));
    int *const lens = ints(tensor(a[1], "lens"), "lens", s.device, {s.rows});
    const Tensor &rows = tensor(a[3], "rows");
    const int count = as_int(rows.numel(), "the number of rows");
    const int *r = ints(rows, "rows", s.device, {count});
    const c10::cuda::CUDAGuard guard(s.device);
    const int rc = count == 0 ? ATTN_OK
                              : attn_pages_free(s.table, lens, s.refs, r, count, s.rows, s.pages, s.width,
                                                stream_of(s.device));
    if (rc != ATTN_OK) return status(rc);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// pages_compact(k_pages, v_pages, page_table, refs, table_out, refs_out, workspace)
PyObject *pages_compact(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_args(n, 7)) return nullptr;
    const Pools p(tensor(a[0], "k_pages"), maybe(a[1], "v_pages"));
    const State s(tensor(a[2], "page_table"), tensor(a[3], "refs"));
    TORCH_CHECK_VALUE(s.device == p.device && s.pages == p.pages,
                      "refs must have one count a page, on the pages' device");
    int *const table_out = ints(tensor(a[4], "the table in out"), "the table in out", p.device, {s.rows, s.width});
    int *const refs_out = ints(tensor(a[5], "the counts in out"), "the counts in out", p.device, {s.pages});
    const c10::cuda::CUDAGuard guard(p.device);
    Tensor live = fresh({1}, at::kInt, p.device);
    const Tensor &given = maybe(a[6], "workspace");
    const Scratch w(given, given.defined() ? 0 : attn_pages_workspace_bytes(0, s.rows, s.pages),
                    "the page operations", p.device);
    const int rc = attn_pages_compact(p.k, p.v, p.strides.ptr, s.table, s.refs, table_out, refs_out,
                                      live.data_ptr<int>(), w.ptr, w.bytes, s.rows, p.heads, p.pages, p.page_size,
                                      s.width, p.d, stream_of(p.device));
    return rc == ATTN_OK ? THPVariable_Wrap(std::move(live)) : status(rc);
    END_HANDLE_TH_ERRORS
}

#define ATTN_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ATTN_METHOD(decode_paged),  ATTN_METHOD(decode_latent), ATTN_METHOD(pages_append),
                         ATTN_METHOD(pages_reserve), ATTN_METHOD(pages_fork),    ATTN_METHOD(pages_free),
                         ATTN_METHOD(pages_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "attn_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit_attn_bind() { return PyModule_Create(&module); }
