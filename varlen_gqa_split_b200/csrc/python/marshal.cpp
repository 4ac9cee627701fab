// marshal.cpp -- argument marshalling of the cache operators (rope, append, key
// weights, eviction): checks the types, shapes, strides and devices of the
// tensors it is given and calls libvgqa's C ABI with their addresses.  A decode
// step calls these operators once a layer with ten tensors each; reading the
// tensors' attributes and converting two dozen arguments from Python took 7 to
// 15 us of host time a call, more than the smallest kernels run.
#include <Python.h>
#include <dlfcn.h>
#include <stdint.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <initializer_list>

#include "../../../include/varlen_gqa.h"

namespace {

decltype(&attn_rope_apply) f_rope;
decltype(&attn_append_paged) f_append;
decltype(&attn_key_weights) f_weights;
decltype(&attn_key_weights_paged) f_weights_paged;
decltype(&attn_evict_paged) f_evict;

// thrown after a Python error was set
struct Refused {};

template <typename... A>
[[noreturn]] void refuse(PyObject *type, const char *format, A... args) {
    PyErr_Format(type, format, args...);
    throw Refused{};
}

long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

void *address(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused{};
    return p;
}

const at::Tensor &tensor(PyObject *o, const char *name, at::ScalarType type, long long dev) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != type) refuse(PyExc_ValueError, "%s must be of type %s", name, c10::toString(type));
    if (!t.is_cuda() || t.get_device() != dev) refuse(PyExc_ValueError, "%s must be on CUDA device %lld", name, dev);
    return t;
}

// [T, H, D] with the heads contiguous within a token; *stride is the tokens' (a
// single token has none that matters)
void *heads(PyObject *o, const char *name, at::ScalarType type, long long dev, long long T, long long H, long long D,
            long long *stride) {
    const at::Tensor &t = tensor(o, name, type, dev);
    if (t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != D)
        refuse(PyExc_ValueError, "%s must be [%lld, %lld, %lld]", name, T, H, D);
    if ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D))
        refuse(PyExc_ValueError, "%s must keep each token's heads contiguous (strides (s, D, 1), s >= H*D)", name);
    *stride = T > 1 ? (long long)t.stride(0) : H * D;
    return t.data_ptr();
}

// a contiguous tensor of a given shape
void *packed(PyObject *o, const char *name, at::ScalarType type, long long dev, at::IntArrayRef shape) {
    const at::Tensor &t = tensor(o, name, type, dev);
    if (t.sizes() != shape || !t.is_contiguous()) {
        if (shape.size() == 3)
            refuse(PyExc_ValueError, "%s must be a contiguous [%lld, %lld, %lld]", name, (long long)shape[0],
                   (long long)shape[1], (long long)shape[2]);
        refuse(PyExc_ValueError, "%s must be a contiguous [%lld, %lld]", name, (long long)shape[0], (long long)shape[1]);
    }
    return t.data_ptr();
}

int32_t *per_sequence(PyObject *o, const char *name, long long dev, long long n) {
    const at::Tensor &t = tensor(o, name, at::kInt, dev);
    if (t.numel() != n || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous int32 tensor of %lld entries", name, n);
    return t.data_ptr<int32_t>();
}

// pos [n_axes, T], or [T] for one axis
const int32_t *positions(PyObject *o, long long dev, long long n_axes, long long T, long long *stride) {
    const at::Tensor &t = tensor(o, "pos", at::kInt, dev);
    if (t.dim() == 1 && n_axes == 1 && t.size(0) == T && (T <= 1 || t.stride(0) == 1)) {
        *stride = T;
    } else {
        if (t.dim() != 2 || t.size(0) != n_axes || t.size(1) != T || (T > 1 && t.stride(1) != 1))
            refuse(PyExc_ValueError, "pos must be [%lld, %lld], unit stride over tokens", n_axes, T);
        *stride = n_axes > 1 ? t.stride(0) : T;
    }
    return t.data_ptr<int32_t>();
}

struct PlanArgs {
    attn_plan_t plan;
    long long B, Hq, Hkv, D, dev, s_max;
    explicit PlanArgs(PyObject *o) {
        plan = static_cast<attn_plan_t>(address(PyTuple_GET_ITEM(o, 0)));
        long long *dst[] = {&B, &Hq, &Hkv, &D, &dev, &s_max};
        for (int i = 0; i < 6; ++i) *dst[i] = integer(PyTuple_GET_ITEM(o, i + 1));
    }
};

// the cache arguments of the paged entry points
struct CacheArgs {
    void *k = nullptr, *v = nullptr;
    long long page_stride, token_stride;
    int page_size, num_pages, bt_stride;
    const int32_t *table;
    CacheArgs(const PlanArgs &p, PyObject *ko, PyObject *vo, PyObject *to) {
        const at::Tensor &kc = tensor(ko, "k_cache", at::kBFloat16, p.dev);
        if (kc.dim() != 4 || kc.size(2) != p.Hkv || kc.size(3) != p.D)
            refuse(PyExc_ValueError, "k_cache must be [num_pages, page_size, %lld, %lld]", p.Hkv, p.D);
        if (kc.stride(3) != 1 || (p.Hkv > 1 && kc.stride(2) != p.D))
            refuse(PyExc_ValueError, "k_cache must keep each token's heads contiguous");
        if (vo) {
            const at::Tensor &vc = tensor(vo, "v_cache", at::kBFloat16, p.dev);
            if (vc.sizes() != kc.sizes() || vc.strides() != kc.strides())
                refuse(PyExc_ValueError, "k_cache and v_cache must have the same shape and strides");
            v = vc.data_ptr();
        }
        k = kc.data_ptr();
        if (kc.size(0) > INT32_MAX || kc.size(1) > INT32_MAX)
            refuse(PyExc_ValueError, "the cache has too many pages");
        num_pages = (int)kc.size(0);
        page_size = (int)kc.size(1);
        token_stride = page_size > 1 ? kc.stride(1) : p.Hkv * p.D;
        page_stride = num_pages > 1 ? kc.stride(0) : page_size * token_stride;
        const at::Tensor &bt = tensor(to, "block_table", at::kInt, p.dev);
        if (bt.dim() != 2 || bt.size(0) != p.B || (bt.size(1) > 1 && bt.stride(1) != 1))
            refuse(PyExc_ValueError, "block_table must be [%lld, n] with unit column stride", p.B);
        if (bt.size(1) * page_size < p.s_max) refuse(PyExc_ValueError, "block_table rows must cover s_max keys");
        const long long s = p.B > 1 ? bt.stride(0) : std::max<long long>(bt.stride(0), bt.size(1));
        if (s > INT32_MAX) refuse(PyExc_ValueError, "block_table rows are too far apart");
        bt_stride = (int)s;
        table = bt.data_ptr<int32_t>();
    }
};

bool given(PyObject *o) { return o != Py_None; }

// The C ABI call without the interpreter lock, its code as a Python integer.
// `written` (tensors or None) count as changed in place, so that autograd
// notices where it had saved one.
template <typename F> PyObject *call(std::initializer_list<PyObject *> written, F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = f();
    Py_END_ALLOW_THREADS
    if (rc == ATTN_OK)
        for (PyObject *o : written)
            if (given(o)) {
                const at::Tensor &t = THPVariable_Unpack(o);
                if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
            }
    return PyLong_FromLong(rc);
}

template <typename F> PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    try {
        if (n != want) refuse(PyExc_TypeError, "takes %zd arguments", want);
        return f();
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (handle, D, n_axes, device, x, pos, out, grad, stream)
PyObject *rope_apply(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const auto rope = static_cast<attn_rope_t>(address(a[0]));
        const long long D = integer(a[1]), dev = integer(a[3]);
        if (!THPVariable_Check(a[4])) refuse(PyExc_TypeError, "x must be a tensor");
        const at::Tensor &x = THPVariable_Unpack(a[4]);
        const at::ScalarType type = x.scalar_type();
        const int dtype = type == at::kBFloat16 ? ATTN_DTYPE_BF16 : type == at::kHalf ? ATTN_DTYPE_F16 : ATTN_DTYPE_F32;
        if (dtype == ATTN_DTYPE_F32 && type != at::kFloat) refuse(PyExc_TypeError, "x must be bf16, fp16 or fp32");
        if (x.dim() != 3) refuse(PyExc_ValueError, "x must be [T, H, D]");
        const long long T = x.size(0), H = x.size(1);
        long long xs, os, ps;
        void *xp = heads(a[4], "x", type, dev, T, H, D, &xs);
        void *op = heads(a[6], "out", type, dev, T, H, D, &os);
        const int32_t *pos = positions(a[5], dev, integer(a[2]), T, &ps);
        const int grad = PyObject_IsTrue(a[7]);
        void *stream = address(a[8]);
        if (T == 0 || H == 0) return PyLong_FromLong(0);
        if (H > INT32_MAX) refuse(PyExc_ValueError, "x has too many heads");
        return call({a[6]}, [&] { return f_rope(rope, dtype, xp, xs, T, (int)H, pos, ps, grad, op, os, stream); });
    });
}

// (plan, rope or 0, n_axes, k, v, k_cache, v_cache, block_table, cu_q, cu_k, q, pos, q_out, stream)
PyObject *append_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        const PlanArgs p(a[0]);
        const auto rope = static_cast<attn_rope_t>(address(a[1]));
        const at::Tensor &k0 = tensor(a[3], "k", at::kBFloat16, p.dev);
        const long long T = k0.dim() ? k0.size(0) : 0;
        long long ks, vs, qs = 0, ps = 0;
        void *k = heads(a[3], "k", at::kBFloat16, p.dev, T, p.Hkv, p.D, &ks);
        void *v = heads(a[4], "v", at::kBFloat16, p.dev, T, p.Hkv, p.D, &vs);
        void *q = nullptr, *q_out = nullptr;
        if (given(a[10])) {
            q = heads(a[10], "q", at::kBFloat16, p.dev, T, p.Hq, p.D, &qs);
            q_out = packed(a[12], "q_out", at::kBFloat16, p.dev, {T, p.Hq, p.D});
        }
        const int32_t *pos = rope ? positions(a[11], p.dev, integer(a[2]), T, &ps) : nullptr;
        const CacheArgs c(p, a[5], a[6], a[7]);
        const int32_t *cu_q = per_sequence(a[8], "cu_q", p.dev, p.B + 1), *cu_k = per_sequence(a[9], "cu_k", p.dev, p.B + 1);
        void *stream = address(a[13]);
        if (T == 0) return PyLong_FromLong(0);
        return call({a[5], a[6], a[12]}, [&] {
            return f_append(p.plan, rope, q, qs, k, ks, v, vs, T, pos, ps, q_out, c.k, c.v, c.page_stride, c.token_stride,
                            c.page_size, c.num_pages, c.table, c.bt_stride, cu_q, cu_k, stream);
        });
    });
}

// (plan, q, k or k_cache, block_table or None, cu_q, cu_k, lse, weight_in, decay, out, seen, born, stream)
PyObject *key_weights(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject * {
        const PlanArgs p(a[0]);
        const at::Tensor &q0 = tensor(a[1], "q", at::kBFloat16, p.dev);
        const long long T = q0.dim() ? q0.size(0) : 0;
        void *q = packed(a[1], "q", at::kBFloat16, p.dev, {T, p.Hq, p.D});
        const auto *lse = static_cast<const float *>(packed(a[6], "lse", at::kFloat, p.dev, {T, p.Hq}));
        const at::Tensor &o = tensor(a[9], "out", at::kFloat, p.dev);
        if (o.dim() != 3 || o.size(0) != p.B || o.size(1) != p.Hkv || o.size(2) < p.s_max)
            refuse(PyExc_ValueError, "out must be [%lld, %lld, >= %lld]", p.B, p.Hkv, p.s_max);
        const long long ld = o.size(2);
        const at::IntArrayRef shape = o.sizes();
        auto *out = static_cast<float *>(packed(a[9], "out", at::kFloat, p.dev, shape));
        const float *in = given(a[7]) ? static_cast<const float *>(packed(a[7], "weight_in", at::kFloat, p.dev, shape)) : nullptr;
        if (given(a[10]) != given(a[11])) refuse(PyExc_ValueError, "seen and born go together");
        const int32_t *seen = given(a[10]) ? per_sequence(a[10], "seen", p.dev, p.B) : nullptr;
        auto *born = given(a[11]) ? static_cast<int32_t *>(packed(a[11], "born", at::kInt, p.dev, shape)) : nullptr;
        const int32_t *cu_q = per_sequence(a[4], "cu_q", p.dev, p.B + 1), *cu_k = per_sequence(a[5], "cu_k", p.dev, p.B + 1);
        const double decay = PyFloat_AsDouble(a[8]);
        if (decay == -1.0 && PyErr_Occurred()) throw Refused{};
        void *stream = address(a[12]);
        if (given(a[3])) {
            const CacheArgs c(p, a[2], nullptr, a[3]);
            return call({a[9], a[11]}, [&] {
                return f_weights_paged(p.plan, q, T, c.k, c.page_stride, c.token_stride, c.page_size, c.num_pages, c.table,
                                       c.bt_stride, cu_q, cu_k, lse, (float)decay, in, out, ld, seen, born, stream);
            });
        }
        const at::Tensor &k0 = tensor(a[2], "k", at::kBFloat16, p.dev);
        long long ks;
        const long long T_kv = k0.dim() ? k0.size(0) : 0;
        void *k = heads(a[2], "k", at::kBFloat16, p.dev, T_kv, p.Hkv, p.D, &ks);
        return call({a[9], a[11]}, [&] {
            return f_weights(p.plan, q, T, k, ks, T_kv, cu_q, cu_k, lse, (float)decay, in, out, ld, seen, born, stream);
        });
    });
}

// (plan, weight, born, seen, keep, k_cache, v_cache, block_table, cu_k, sink, recent, weight_out, born_out, cu_k_out,
// stream)
PyObject *evict_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        const PlanArgs p(a[0]);
        const at::Tensor &w0 = tensor(a[1], "weight", at::kFloat, p.dev);
        if (w0.dim() != 3 || w0.size(0) != p.B || w0.size(1) != p.Hkv || w0.size(2) < p.s_max)
            refuse(PyExc_ValueError, "weight must be [%lld, %lld, >= %lld]", p.B, p.Hkv, p.s_max);
        const at::IntArrayRef shape = w0.sizes();
        auto ledger = [&](int i, const char *name, at::ScalarType type) { return packed(a[i], name, type, p.dev, shape); };
        const auto *w = static_cast<const float *>(ledger(1, "weight", at::kFloat));
        const auto *born = static_cast<const int32_t *>(ledger(2, "born", at::kInt));
        auto *w_out = static_cast<float *>(ledger(11, "weight_out", at::kFloat));
        auto *born_out = static_cast<int32_t *>(ledger(12, "born_out", at::kInt));
        const CacheArgs c(p, a[5], a[6], a[7]);
        const int32_t *seen = per_sequence(a[3], "seen", p.dev, p.B), *keep = per_sequence(a[4], "keep", p.dev, p.B);
        const int32_t *cu_k = per_sequence(a[8], "cu_k", p.dev, p.B + 1);
        int32_t *cu_out = per_sequence(a[13], "cu_k_out", p.dev, p.B + 1);
        const long long sink = integer(a[9]), recent = integer(a[10]);
        if (sink > INT32_MAX || recent > INT32_MAX || sink < 0 || recent < 0)
            refuse(PyExc_ValueError, "sink and recent must be in [0, 2^31)");
        void *stream = address(a[14]);
        return call({a[5], a[6], a[11], a[12], a[13]}, [&] {
            return f_evict(p.plan, w, born, seen, keep, (int)sink, (int)recent, w_out, born_out, shape[2], c.k, c.v,
                           c.page_stride, c.token_stride, c.page_size, c.num_pages, c.table, c.bt_stride, cu_k, cu_out,
                           stream);
        });
    });
}

// bind(path): the library whose entry points are called
PyObject *bind(PyObject *, PyObject *path) {
    const char *name = PyUnicode_AsUTF8(path);
    if (!name) return nullptr;
    void *h = dlopen(name, RTLD_NOW);
    if (!h) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    f_rope = reinterpret_cast<decltype(f_rope)>(dlsym(h, "attn_rope_apply"));
    f_append = reinterpret_cast<decltype(f_append)>(dlsym(h, "attn_append_paged"));
    f_weights = reinterpret_cast<decltype(f_weights)>(dlsym(h, "attn_key_weights"));
    f_weights_paged = reinterpret_cast<decltype(f_weights_paged)>(dlsym(h, "attn_key_weights_paged"));
    f_evict = reinterpret_cast<decltype(f_evict)>(dlsym(h, "attn_evict_paged"));
    if (!f_rope || !f_append || !f_weights || !f_weights_paged || !f_evict) {
        PyErr_SetString(PyExc_RuntimeError, "the library lacks an entry point of the cache operators");
        return nullptr;
    }
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"rope_apply", (PyCFunction)(void (*)())rope_apply, METH_FASTCALL, nullptr},
                         {"append_paged", (PyCFunction)(void (*)())append_paged, METH_FASTCALL, nullptr},
                         {"key_weights", (PyCFunction)(void (*)())key_weights, METH_FASTCALL, nullptr},
                         {"evict_paged", (PyCFunction)(void (*)())evict_paged, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
