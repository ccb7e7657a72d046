// Python calls of libcsa.so's paged cache and rotary positions (include/csa.h)
// on torch tensors, as a CPython module: _paged.py holds their signatures and
// documentation.
//
// Argument marshalling only: tensors are checked for device, dtype, shape and
// layout (ValueError), outputs are taken from torch's allocator, and pointers
// and torch's current stream on the tensors' device go to the C entry point,
// whose status becomes a CsaError.  In C++ because these calls are short: the
// kernels of a decode step take 3 to 10 us each, the same checks and two
// outputs in Python 13 to 20 us, here 2 to 3 us.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <initializer_list>

#include "csa.h"

namespace {

using at::IntArrayRef;
using at::Tensor;

PyObject *g_error = nullptr;  // CsaError

void check(int status, const char *where) {
    if (status == CSA_OK) return;
    if (PyObject *e = PyObject_CallFunction(g_error, "is", status, where)) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

const Tensor &tensor(PyObject *o, const char *name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

const Tensor *optional(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

int integer(PyObject *o, const char *name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, name, " out of range: ", v);
    return (int)v;
}

int size(int64_t n, const char *name) {
    TORCH_CHECK_VALUE(n <= INT_MAX, name, " out of range: ", n);
    return (int)n;
}

void need_kind(const Tensor &t, const char *name, at::ScalarType dtype, IntArrayRef shape, const at::Device &dev) {
    TORCH_CHECK_VALUE(t.device() == dev, name, " must be on ", dev, ", got ", t.device());
    TORCH_CHECK_VALUE(t.scalar_type() == dtype, name, " must be ", dtype, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
}

void need(const Tensor &t, const char *name, at::ScalarType dtype, IntArrayRef shape, const at::Device &dev) {
    need_kind(t, name, dtype, shape, dev);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}

// The allocator's tensor without the dispatcher's two hops: 0.2 us less each (rope with two outputs
// 5.2 -> 5.0 us a call, 2.7 with given ones).  Hooks of the dispatcher do not see it, as they do not
// see the kernels; the allocator's own statistics do.
Tensor made(IntArrayRef shape, at::ScalarType dtype, const at::Device &dev) {
    return Tensor(at::detail::empty_cuda(shape, dtype, dev, std::nullopt));
}

// The given output, checked, or a new one.
Tensor out(const Tensor *given, const char *name, at::ScalarType dtype, IntArrayRef shape, const at::Device &dev) {
    if (!given) return made(shape, dtype, dev);
    need(*given, name, dtype, shape, dev);
    return *given;
}

template <typename T = void>
T *at_(const Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}
template <typename T = void>
T *at_(const Tensor *t) {
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}

// What a call has written: autograd compares versions to see that a saved tensor has not changed since.
void wrote(std::initializer_list<const Tensor *> written) {
    for (const Tensor *t : written)
        if (t && t->defined() && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// The device of the call: the first tensor's, made the current one.
struct Here {
    at::Device dev;
    c10::cuda::OptionalCUDAGuard guard;
    csa_stream_t stream;
    explicit Here(const Tensor &t, const char *what) : dev(t.device()) {
        TORCH_CHECK_VALUE(dev.is_cuda(), what, " takes CUDA tensors");
        guard.set_device(dev);
        stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
};

PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

PyObject *tuple(std::initializer_list<Tensor> items) {
    PyObject *r = PyTuple_New((Py_ssize_t)items.size());
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor &t : items) {
        PyObject *o;
        if (t.defined()) {
            o = wrap(t);
        } else {
            Py_INCREF(Py_None);
            o = Py_None;
        }
        if (!o) {
            Py_DECREF(r);
            throw python_error();
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// ------------------------------------------------------------------ decode
// q, k_pages, v_pages, block_table, seqlens, k0, v0, mode, scale, out, lse, workspace, want_lse
PyObject *decode_paged(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_pages"), &v = tensor(a[2], "v_pages"),
                 &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seqlens");
    Here here(q, "decode_paged");
    TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() == 4 && table.dim() == 2,
                      "q is [B, Hq, d], the pools [P, Hkv, S, d], block_table [B, M]");
    const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2), P = k.size(0), Hkv = k.size(1), S = k.size(2),
                  M = table.size(1);
    const auto bf = at::kBFloat16;
    need(q, "q", bf, {B, Hq, d}, here.dev);
    need(k, "k_pages", bf, {P, Hkv, S, d}, here.dev);
    need(v, "v_pages", bf, {P, Hkv, S, d}, here.dev);
    need(table, "block_table", at::kInt, {B, M}, here.dev);
    need(lens, "seqlens", at::kInt, {B}, here.dev);
    const int mode = integer(a[7], "mode");
    const Tensor *k0 = nullptr, *v0 = nullptr;
    if (mode == CSA_K0_GIVEN) {
        k0 = optional(a[5], "k0");
        v0 = optional(a[6], "v0");
        TORCH_CHECK_VALUE(k0 && v0, "mode 2 (given sink) needs k0 and v0");
        need(*k0, "k0", bf, {Hkv, d}, here.dev);
        need(*v0, "v0", bf, {Hkv, d}, here.dev);
    }
    double scale = 1.0 / std::sqrt((double)d);
    if (a[8] != Py_None) {
        scale = PyFloat_AsDouble(a[8]);
        if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    }
    Tensor o = out(optional(a[9], "out"), "out", bf, {B, Hq, d}, here.dev), lse;
    const Tensor *lse_given = optional(a[10], "lse");
    const int want_lse = PyObject_IsTrue(a[12]);
    if (want_lse < 0) throw python_error();
    if (lse_given || want_lse) lse = out(lse_given, "lse", at::kFloat, {B, Hq}, here.dev);
    const int b = size(B, "B"), hq = size(Hq, "Hq"), hkv = size(Hkv, "Hkv"), dd = size(d, "d");
    const Tensor *ws = optional(a[11], "workspace");
    Tensor own;
    if (!ws) {
        own = made({std::max<long long>(csa_decode_paged_workspace_bytes(b, hq, hkv, dd), 16)}, at::kByte, here.dev);
        ws = &own;
    }
    TORCH_CHECK_VALUE(ws->device() == here.dev && ws->is_contiguous(), "workspace must be a contiguous tensor on ",
                      here.dev);
    check(csa_decode_paged(at_(q), at_(k), at_(v), at_(k0), at_(v0), at_<int>(table), at_<int>(lens), at_(o),
                           lse.defined() ? at_<float>(lse) : nullptr, at_(ws), (long long)ws->nbytes(), b, hq, hkv,
                           size(P, "P"), size(S, "S"), size(M, "M"), dd, (float)scale, mode, here.stream),
          "csa_decode_paged");
    wrote({&o, &lse, ws});
    return tuple({o, lse});
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ rotary positions
// A tensor of rows [B, H, T, d] whose last dimension is contiguous: its
// strides over batch, head and time.
struct Rows {
    long long strides[3];
    Rows(const Tensor &t, const char *name, at::ScalarType dtype, IntArrayRef shape, const at::Device &dev,
         bool written) {
        need_kind(t, name, dtype, shape, dev);
        const IntArrayRef s = t.strides();
        TORCH_CHECK_VALUE(s[3] == 1 || shape[3] <= 1, "the last dimension of ", name, " must be contiguous");
        for (int i = 0; i < 3; ++i) strides[i] = s[i];
        if (written && !t.is_contiguous()) {
            std::pair<int64_t, int64_t> dims[3];
            for (int i = 0; i < 3; ++i) dims[i] = {s[i], shape[i]};
            std::sort(dims, dims + 3);
            int64_t reach = shape[3];
            for (const auto &[stride, n] : dims)
                if (n > 1) {
                    TORCH_CHECK_VALUE(stride >= reach, "rows of ", name, " overlap");
                    reach += stride * (n - 1);
                }
        }
    }
    Rows() = default;
};

// positions: [axes, B, T], or [B, T] or [T] with one axis
void position_strides(const Tensor &t, int axes, int64_t B, int64_t T, const at::Device &dev, long long (&strides)[3]) {
    TORCH_CHECK_VALUE(t.device() == dev && t.scalar_type() == at::kInt, "positions must be int32 on ", dev, ", got ",
                      t.scalar_type(), " on ", t.device());
    const IntArrayRef n = t.sizes(), s = t.strides();
    strides[0] = strides[1] = strides[2] = 0;
    if (n.size() == 3 && n[0] == axes && n[1] == B && n[2] == T) {
        for (int i = 0; i < 3; ++i) strides[i] = s[i];
    } else if (axes == 1 && n.size() == 2 && n[0] == B && n[1] == T) {
        strides[1] = s[0];
        strides[2] = s[1];
    } else if (axes == 1 && n.size() == 1 && n[0] == T) {
        strides[2] = s[0];
    } else {
        TORCH_CHECK_VALUE(false, "positions must have shape [", axes, ", ", B, ", ", T, "]",
                          axes == 1 ? " (or without its first dimensions)" : "", ", got ", n);
    }
}

const csa_rope_plan *plan_at(PyObject *address) {
    void *p = PyLong_AsVoidPtr(address);
    if (!p && PyErr_Occurred()) throw python_error();
    return static_cast<const csa_rope_plan *>(p);
}

bool is_bf16(at::ScalarType dtype) {
    TORCH_CHECK_VALUE(dtype == at::kBFloat16 || dtype == at::kFloat, "unsupported dtype ", dtype);
    return dtype == at::kBFloat16;
}

// q, k, positions, plan address, plan d, q_out, k_out, inverse
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &q = tensor(a[0], "q"), &positions = tensor(a[2], "positions");
    const Tensor *k = optional(a[1], "k");
    Here here(q, "rope");
    TORCH_CHECK_VALUE(q.dim() == 4 && (!k || k->dim() == 4), "q and k are [B, H, T, d]");
    const int64_t B = q.size(0), Hq = q.size(1), T = q.size(2), d = q.size(3), Hkv = k ? k->size(1) : 0;
    const auto dtype = q.scalar_type();
    const bool bf = is_bf16(dtype);
    const csa_rope_plan *plan = plan_at(a[3]);
    TORCH_CHECK_VALUE(integer(a[4], "d") == d, "the plan is for rows of ", integer(a[4], "d"), ", got ", d);
    long long ps[3];
    position_strides(positions, plan->axes, B, T, here.dev, ps);
    const Rows qs(q, "q", dtype, {B, Hq, T, d}, here.dev, false);
    const Tensor *given = optional(a[5], "q_out");
    const Tensor qo = given ? *given : made({B, Hq, T, d}, dtype, here.dev);
    const Rows qos(qo, "q_out", dtype, {B, Hq, T, d}, here.dev, true);
    Rows ks, kos;
    Tensor ko;
    TORCH_CHECK_VALUE(k || a[6] == Py_None, "k_out goes with k");
    if (k) {
        ks = Rows(*k, "k", dtype, {B, Hkv, T, d}, here.dev, false);
        given = optional(a[6], "k_out");
        ko = given ? *given : made({B, Hkv, T, d}, dtype, here.dev);
        kos = Rows(ko, "k_out", dtype, {B, Hkv, T, d}, here.dev, true);
    }
    const int b = size(B, "B"), hq = size(Hq, "Hq"), hkv = size(Hkv, "Hkv"), t = size(T, "T"), dd = size(d, "d");
    const int inverse = integer(a[7], "inverse");
    void *kp = at_(k), *kop = k ? at_(ko) : nullptr;
    if (bf)
        check(csa_rope(plan, at_(q), qs.strides, at_(qo), qos.strides, kp, ks.strides, kop, kos.strides,
                       at_<int>(positions), ps, b, hq, hkv, t, dd, inverse, here.stream),
              "csa_rope");
    else
        check(csa_rope_f32(plan, at_<float>(q), qs.strides, at_<float>(qo), qos.strides, static_cast<float *>(kp),
                           ks.strides, static_cast<float *>(kop), kos.strides, at_<int>(positions), ps, b, hq, hkv, t,
                           dd, inverse, here.stream),
              "csa_rope_f32");
    wrote({&qo, &ko});
    return tuple({qo, ko});
    END_HANDLE_TH_ERRORS
}

// k, v, k_pages, v_pages, block_table, seqlens, counts, plan address or None, plan d, positions, q, q_out
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &kp = tensor(a[2], "k_pages"),
                 &vp = tensor(a[3], "v_pages"), &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "seqlens");
    Here here(k, "cache_append");
    TORCH_CHECK_VALUE(k.dim() == 4 && kp.dim() == 4 && table.dim() == 2,
                      "k and v are [B, Hkv, T, d], the pools [P, Hkv, S, d], block_table [B, M]");
    const int64_t B = k.size(0), Hkv = k.size(1), T = k.size(2), d = k.size(3), P = kp.size(0), S = kp.size(2),
                  M = table.size(1);
    const auto dtype = k.scalar_type();
    const bool bf = is_bf16(dtype);
    const Rows ks(k, "k", dtype, {B, Hkv, T, d}, here.dev, false), vs(v, "v", dtype, {B, Hkv, T, d}, here.dev, false);
    need(kp, "k_pages", dtype, {P, Hkv, S, d}, here.dev);
    need(vp, "v_pages", dtype, {P, Hkv, S, d}, here.dev);
    need(table, "block_table", at::kInt, {B, M}, here.dev);
    need(lens, "seqlens", at::kInt, {B}, here.dev);
    const Tensor *counts = optional(a[6], "counts"), *positions = optional(a[9], "positions"), *q = optional(a[10], "q");
    if (counts) need(*counts, "counts", at::kInt, {B}, here.dev);
    const csa_rope_plan *plan = nullptr;
    long long ps[3] = {0, 0, 0};
    int64_t Hq = 0;
    Rows qs, qos;
    Tensor qo;
    TORCH_CHECK_VALUE(q || a[11] == Py_None, "q_out goes with q");
    if (a[7] == Py_None) {
        TORCH_CHECK_VALUE(!q && !positions, "q and positions go with a rope plan");
    } else {
        plan = plan_at(a[7]);
        TORCH_CHECK_VALUE(integer(a[8], "d") == d, "the plan is for rows of ", integer(a[8], "d"), ", got ", d);
        if (positions) position_strides(*positions, plan->axes, B, T, here.dev, ps);
        if (q) {
            TORCH_CHECK_VALUE(q->dim() == 4, "q is [B, Hq, T, d]");
            Hq = q->size(1);
            qs = Rows(*q, "q", dtype, {B, Hq, T, d}, here.dev, false);
            const Tensor *given = optional(a[11], "q_out");
            qo = given ? *given : made({B, Hq, T, d}, dtype, here.dev);
            qos = Rows(qo, "q_out", dtype, {B, Hq, T, d}, here.dev, true);
        }
    }
    const int b = size(B, "B"), hq = size(Hq, "Hq"), hkv = size(Hkv, "Hkv"), t = size(T, "T"), dd = size(d, "d"),
              pp = size(P, "P"), ss = size(S, "S"), m = size(M, "M");
    void *qp = at_(q), *qop = qo.defined() ? at_(qo) : nullptr;
    if (bf)
        check(csa_cache_append(plan, qp, qs.strides, qop, qos.strides, at_(k), ks.strides, at_(v), vs.strides, at_(kp),
                               at_(vp), at_<int>(table), at_<int>(lens), at_<int>(counts), at_<int>(positions), ps, b,
                               hq, hkv, t, dd, pp, ss, m, here.stream),
              "csa_cache_append");
    else
        check(csa_cache_append_f32(plan, static_cast<float *>(qp), qs.strides, static_cast<float *>(qop), qos.strides,
                                   at_<float>(k), ks.strides, at_<float>(v), vs.strides, at_<float>(kp),
                                   at_<float>(vp), at_<int>(table), at_<int>(lens), at_<int>(counts),
                                   at_<int>(positions), ps, b, hq, hkv, t, dd, pp, ss, m, here.stream),
              "csa_cache_append_f32");
    wrote({&kp, &vp, &qo});
    if (!qo.defined()) Py_RETURN_NONE;
    return wrap(qo);
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------ pages
struct Books {
    Here here;
    const Tensor &t_refs, &t_table, &t_lens;
    int *refs, *table, *lens;
    int P, B, M, S;
    // page_refs, block_table, seqlens, page_size
    Books(PyObject *const *a, const char *what)
        : here(tensor(a[0], "page_refs"), what), t_refs(tensor(a[0], "page_refs")),
          t_table(tensor(a[1], "block_table")), t_lens(tensor(a[2], "seqlens")) {
        const Tensor &r = t_refs, &t = t_table, &n = t_lens;
        TORCH_CHECK_VALUE(r.dim() == 1 && t.dim() == 2, "page_refs is [P], block_table [B, M]");
        need(r, "page_refs", at::kInt, {r.size(0)}, here.dev);
        need(t, "block_table", at::kInt, {t.size(0), t.size(1)}, here.dev);
        need(n, "seqlens", at::kInt, {t.size(0)}, here.dev);
        P = size(r.size(0), "P");
        B = size(t.size(0), "B");
        M = size(t.size(1), "M");
        S = integer(a[3], "page_size");
        refs = at_<int>(r);
        table = at_<int>(t);
        lens = at_<int>(n);
    }
};

// ..., counts, shortfall
PyObject *cache_reserve(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Books b(a, "cache_reserve");
    const Tensor &counts = tensor(a[4], "counts");
    need(counts, "counts", at::kInt, {b.B}, b.here.dev);
    Tensor shortfall = out(optional(a[5], "shortfall"), "shortfall", at::kInt, {1}, b.here.dev);
    check(csa_cache_reserve(b.refs, b.table, b.lens, at_<int>(counts), at_<int>(shortfall), b.B, b.P, b.S, b.M,
                            b.here.stream),
          "csa_cache_reserve");
    wrote({&b.t_refs, &b.t_table, &b.t_lens, &shortfall});
    return wrap(shortfall);
    END_HANDLE_TH_ERRORS
}

// ..., rows
PyObject *cache_free(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Books b(a, "cache_free");
    const Tensor &rows = tensor(a[4], "rows");
    need(rows, "rows", at::kInt, {rows.numel()}, b.here.dev);
    check(csa_cache_free(b.refs, b.table, b.lens, at_<int>(rows), size(rows.numel(), "rows"), b.B, b.P, b.S, b.M,
                         b.here.stream),
          "csa_cache_free");
    wrote({&b.t_refs, &b.t_table, &b.t_lens});
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// ..., parents, children
PyObject *cache_fork(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Books b(a, "cache_fork");
    const Tensor &parents = tensor(a[4], "parents"), &children = tensor(a[5], "children");
    const int n = size(parents.numel(), "parents");
    need(parents, "parents", at::kInt, {n}, b.here.dev);
    need(children, "children", at::kInt, {n}, b.here.dev);
    Tensor src = made({n}, at::kInt, b.here.dev), dst = made({n}, at::kInt, b.here.dev),
           shortfall = made({1}, at::kInt, b.here.dev);
    check(csa_cache_fork(b.refs, b.table, b.lens, at_<int>(parents), at_<int>(children), n, at_<int>(src),
                         at_<int>(dst), at_<int>(shortfall), b.B, b.P, b.S, b.M, b.here.stream),
          "csa_cache_fork");
    wrote({&b.t_refs, &b.t_table, &b.t_lens});
    return tuple({src, dst, shortfall});
    END_HANDLE_TH_ERRORS
}

PyObject *cache_compact(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Books b(a, "cache_compact");
    Tensor src = made({b.P / 2}, at::kInt, b.here.dev), dst = made({b.P / 2}, at::kInt, b.here.dev),
           moved = made({1}, at::kInt, b.here.dev);
    check(csa_cache_compact(b.refs, b.table, b.lens, at_<int>(src), at_<int>(dst), at_<int>(moved), b.B, b.P, b.S, b.M,
                            b.here.stream),
          "csa_cache_compact");
    wrote({&b.t_refs, &b.t_table});
    return tuple({src, dst, moved});
    END_HANDLE_TH_ERRORS
}

// k_pages, v_pages, src, dst, count
PyObject *cache_copy_pages(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &k = tensor(a[0], "k_pages"), &src = tensor(a[2], "src"), &dst = tensor(a[3], "dst");
    const Tensor *v = optional(a[1], "v_pages"), *count = optional(a[4], "count");
    Here here(k, "cache_copy_pages");
    TORCH_CHECK_VALUE(k.dim() == 4 || k.dim() == 5, "the pools are [P, Hkv, S, d] or [L, P, Hkv, S, d]");
    need(k, "k_pages", k.scalar_type(), k.sizes(), here.dev);
    if (v) need(*v, "v_pages", k.scalar_type(), k.sizes(), here.dev);
    const int n = size(src.numel(), "src"), layers = k.dim() == 5 ? size(k.size(0), "L") : 1;
    need(src, "src", at::kInt, {n}, here.dev);
    need(dst, "dst", at::kInt, {n}, here.dev);
    if (count) need(*count, "count", at::kInt, {1}, here.dev);
    const long long page = (long long)k.size(-3) * k.size(-2) * k.size(-1) * (long long)k.element_size();
    check(csa_cache_copy_pages(at_(k), at_(v), page, layers, size(k.size(-4), "P"), at_<int>(src), at_<int>(dst), n,
                               at_<int>(count), here.stream),
          "csa_cache_copy_pages");
    wrote({&k, v});
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

// Each function is called by one wrapper of _paged.py, with all of its arguments.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t), int N>
PyObject *counted(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    return F(self, a, n);
}
#define CALL(name, n) {#name, (PyCFunction)(void (*)(void))counted<name, n>, METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {CALL(decode_paged, 13),
                           CALL(rope, 8),
                           CALL(cache_append, 12),
                           CALL(cache_reserve, 6),
                           CALL(cache_free, 5),
                           CALL(cache_fork, 6),
                           CALL(cache_compact, 4),
                           CALL(cache_copy_pages, 5),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_csa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__csa_torch(void) { return PyModule_Create(&g_module); }
