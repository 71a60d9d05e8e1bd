// _rxops: the argument checks and marshalling of the row, page and prompt operators as a Python
// extension: what the binding's Python code does for kv_pool_write_rope, kv_pool_copy,
// kv_pool_fork and prompt_attention, with the same checks and the same library calls, in a
// fraction of the time.  (A decode step's rotary write takes 3 us on the GPU; its 20 arguments cost
// 22 us in the interpreter, 9 us through the tensors' Python methods from C, and 4 us from the
// tensors' C++ fields here.)  No arithmetic of the operators happens here.
//
//   bind({"kv_pool_write_rope": address, ... })
//   kv_pool_write_rope(desc_addr, rope_addr, batch, ..., stream) -> rc        (and the others)
//
// A wrong argument raises ValueError.  stream: None (torch's current stream) or the stream's
// address.  The GIL is released during the native call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>
#include <vector>

#include "radix_attn.h"

namespace {

decltype(&kv_pool_write_rope) g_rope;
decltype(&kv_pool_copy) g_copy;
decltype(&kv_pool_fork) g_fork;
decltype(&prompt_attention) g_prompt;

// A Python exception is set.
struct Raised {};

[[noreturn]] void bad(const std::string& what) {
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Raised{};
}

int64_t as_i64(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

int32_t as_i32(PyObject* o) {
    const int64_t v = as_i64(o);
    if (v < INT32_MIN || v > INT32_MAX) bad(std::to_string(v) + " does not fit 32 bits");
    return (int32_t)v;
}

template <class T>
T* as_ptr(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised{};
    return (T*)p;
}

struct Call {
    const rx_attn_desc* d;
    int64_t dev;
    void* stream;

    Call(PyObject* desc, PyObject* s) : d(as_ptr<const rx_attn_desc>(desc)), dev(c10::cuda::current_device()) {
        stream = s == Py_None ? (void*)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream() : as_ptr<void>(s);
    }

    const at::Tensor& tensor(const char* name, PyObject* o, at::ScalarType type) const {
        if (!THPVariable_Check(o)) bad(std::string(name) + ": want a tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.scalar_type() != type) bad(std::string(name) + ": want " + c10::toString(type));
        if (!t.is_cuda()) bad(std::string(name) + ": not on a CUDA device");
        if (t.get_device() != dev)
            bad(std::string(name) + ": on device " + std::to_string(t.get_device()) + ", but the current device is cuda:" + std::to_string(dev));
        return t;
    }

    at::ScalarType type() const { return d->dtype == RX_F32 ? at::kFloat : at::kBFloat16; }

    // rows [>= total, heads, head_dim] of the descriptor's type, the heads of a row contiguous
    void* rows(const char* name, PyObject* o, int32_t heads, int64_t total, int64_t& stride) const {
        stride = 0;
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(name, o, type());
        const auto sh = t.sizes(), st = t.strides();
        if (sh.size() != 3 || sh[1] != heads || sh[2] != d->head_dim || sh[0] < total || st[2] != 1 || (heads > 1 && st[1] != d->head_dim))
            bad(std::string(name) + ": want [" + std::to_string(total) + ", " + std::to_string(heads) + ", " + std::to_string(d->head_dim) +
                "] with contiguous heads");
        const int64_t row = (int64_t)heads * d->head_dim;
        stride = sh[0] > 1 || st[0] > row ? st[0] : row;
        return t.data_ptr();
    }

    // `count` or more contiguous elements of a type, or a device address as it is
    template <class T>
    T* array(const char* name, PyObject* o, at::ScalarType type, int64_t count) const {
        if (o == Py_None) return nullptr;
        if (PyLong_Check(o)) return as_ptr<T>(o);
        const at::Tensor& t = tensor(name, o, type);
        if (!t.is_contiguous() || t.numel() < count) bad(std::string(name) + ": want " + std::to_string(count) + " contiguous elements");
        return (T*)t.data_ptr();
    }
    int32_t* i32(const char* name, PyObject* o, int64_t count) const { return array<int32_t>(name, o, at::kInt, count); }
    int64_t* i64(const char* name, PyObject* o, int64_t count) const { return array<int64_t>(name, o, at::kLong, count); }

    // a KV pool: contiguous [num_slots, hkv, head_dim]
    void* pool(const char* name, PyObject* o) const {
        const at::Tensor& t = tensor(name, o, type());
        if (!t.is_contiguous() || t.numel() != d->num_slots * d->hkv * d->head_dim)
            bad(std::string(name) + ": want contiguous [" + std::to_string(d->num_slots) + ", " + std::to_string(d->hkv) + ", " +
                std::to_string(d->head_dim) + "]");
        return t.data_ptr();
    }

    std::vector<void*> pools(PyObject* seq) const {
        PyObject* f = PySequence_Fast(seq, "pools: want a sequence of tensors");
        if (!f) throw Raised{};
        struct Ref {
            PyObject* o;
            ~Ref() { Py_DECREF(o); }
        } held{f};
        std::vector<void*> p;
        p.reserve((size_t)PySequence_Fast_GET_SIZE(f) + 1);
        for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(f); ++i) p.push_back(pool("pools", PySequence_Fast_GET_ITEM(f, i)));
        return p;
    }

    // a table [rows, stride] of slots
    int32_t* table(const char* name, PyObject* o, int64_t& n_rows, int64_t& stride) const {
        const at::Tensor& t = tensor(name, o, at::kInt);
        if (t.dim() != 2 || !t.is_contiguous() || t.size(0) > INT32_MAX) bad(std::string(name) + ": want contiguous [rows, stride]");
        n_rows = t.size(0);
        stride = t.size(1);
        return (int32_t*)t.data_ptr();
    }
};

// The call under a released GIL; what is thrown before it becomes a Python exception.
template <class F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, bool bound, F&& f) {
    if (have != want || !bound) {
        PyErr_Format(PyExc_TypeError, bound ? "%zd arguments, got %zd" : "not bound", want, have);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

struct Unlocked {
    PyThreadState* s = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(s); }
};

PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 20, g_rope != nullptr, [&] {
        const Call c(a[0], a[19]);
        const auto* r = as_ptr<const rx_rope_desc>(a[1]);
        const int32_t batch = as_i32(a[2]);
        const int64_t total = as_i64(a[16]);
        int64_t qs, ks, vs, os, xs, ts = 0, unused;
        void* q = c.rows("q", a[8], c.d->hq, total, qs);
        void* k = c.rows("k_new", a[9], c.d->hkv, total, ks);
        void* v = c.rows("v_new", a[10], c.d->hkv, total, vs);
        void* o = c.rows("q_out", a[11], c.d->hq, total, os);
        void* x = c.rows("k_out", a[12], c.d->hkv, total, xs);
        const at::Tensor& pos = c.tensor("positions", a[7], at::kInt);
        if (pos.dim() != 2 || !pos.is_contiguous() || pos.size(0) != r->n_axes || pos.size(1) < total)
            bad("positions: want contiguous [" + std::to_string(r->n_axes) + ", " + std::to_string(total) + "]");
        void* kp = a[5] == Py_None ? nullptr : c.pool("k_pool", a[13]);
        void* vp = a[5] == Py_None ? nullptr : c.pool("v_pool", a[14]);
        if (a[18] != Py_None) ts = as_i64(a[18]);      // the table's stride, where it is given as an address
        else if (a[15] != Py_None) c.table("req_to_token", a[15], unused, ts);
        int32_t* rt = c.i32("req_to_token", a[15], batch * ts);
        const int32_t* ps = c.i32("prefix_slots", a[3], 0);
        const int64_t* pi = c.i64("prefix_indptr", a[4], batch + 1ll);
        const int32_t* ns = c.i32("new_slots", a[5], total);
        const int64_t* qi = c.i64("qo_indptr", a[6], batch + 1ll);
        int32_t* st = c.i32("status", a[17], 1);
        const auto* pp = (const int32_t*)pos.data_ptr();
        const int64_t pstride = pos.size(1);
        Unlocked u;
        return g_rope(c.d, r, batch, ps, pi, ns, qi, pp, pstride, q, qs, k, ks, v, vs, o, os, x, xs, kp, vp, rt, ts, total, st, c.stream);
    });
}

PyObject* py_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, g_copy != nullptr, [&] {
        const Call c(a[0], a[6]);
        const int64_t page = as_i64(a[4]);
        const at::Tensor& src = c.tensor("src", a[2], at::kInt);
        const int64_t count = src.numel();
        if (!src.is_contiguous() || c.tensor("dst", a[3], at::kInt).numel() != count) bad("src, dst: one destination per source");
        const int32_t* dst = c.i32("dst", a[3], count);
        int32_t* st = c.i32("status", a[5], 1);
        std::vector<void*> list = c.pools(a[1]);
        const auto* sp = (const int32_t*)src.data_ptr();
        Unlocked u;
        return g_copy(c.d, (int32_t)list.size(), list.data(), page, count, sp, dst, st, c.stream);
    });
}

PyObject* py_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, g_fork != nullptr, [&] {
        const Call c(a[0], a[11]);
        const int64_t total = as_i64(a[9]);
        int64_t in_rows, in_stride, rows, stride;
        const int32_t* in = c.table("r2t_in", a[7], in_rows, in_stride);
        int32_t* out = c.table("r2t_out", a[8], rows, stride);
        const int32_t* par = c.i32("parents", a[2], rows);
        const int32_t* keep = c.i32("keep_lens", a[3], rows);
        const int32_t* len = c.i32("kv_lens", a[4], rows);
        const int64_t* ti = c.i64("tail_indptr", a[5], rows + 1);
        const int32_t* ts = c.i32("tail_slots", a[6], total);
        int32_t* st = c.i32("status", a[10], 1);
        std::vector<void*> list = c.pools(a[1]);
        Unlocked u;
        return g_fork(c.d, (int32_t)list.size(), list.data(), (int32_t)rows, par, keep, len, ti, ts, in, (int32_t)in_rows, in_stride, out,
                      stride, total, st, c.stream);
    });
}

PyObject* py_prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, g_prompt != nullptr, [&] {
        const Call c(a[0], a[10]);
        const int32_t batch = as_i32(a[1]);
        const int64_t total = as_i64(a[8]);
        int64_t qs, ks, vs, os;
        void* q = c.rows("q", a[2], c.d->hq, total, qs);
        void* k = c.rows("k", a[3], c.d->hkv, total, ks);
        void* v = c.rows("v", a[4], c.d->hkv, total, vs);
        void* o = c.rows("out", a[6], c.d->hq, total, os);
        const int64_t* ip = c.i64("indptr", a[5], batch + 1ll);
        float* lse = c.array<float>("lse", a[7], at::kFloat, total * c.d->hq);
        int32_t* st = c.i32("status", a[9], 1);
        Unlocked u;
        return g_prompt(c.d, batch, q, qs, k, ks, v, vs, ip, o, os, lse, total, st, c.stream);
    });
}

PyObject* py_bind(PyObject*, PyObject* m) {
    void* f[4];
    const char* names[4] = {"kv_pool_write_rope", "kv_pool_copy", "kv_pool_fork", "prompt_attention"};
    for (int i = 0; i < 4; ++i) {
        PyObject* o = PyMapping_GetItemString(m, names[i]);
        if (!o) return nullptr;
        f[i] = PyLong_AsVoidPtr(o);
        Py_DECREF(o);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null function address");
            return nullptr;
        }
    }
    g_rope = (decltype(g_rope))f[0];
    g_copy = (decltype(g_copy))f[1];
    g_fork = (decltype(g_fork))f[2];
    g_prompt = (decltype(g_prompt))f[3];
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"bind", py_bind, METH_O, "Bind the library's functions."},
                         {"kv_pool_write_rope", (PyCFunction)(void (*)())py_rope, METH_FASTCALL, ""},
                         {"kv_pool_copy", (PyCFunction)(void (*)())py_copy, METH_FASTCALL, ""},
                         {"kv_pool_fork", (PyCFunction)(void (*)())py_fork, METH_FASTCALL, ""},
                         {"prompt_attention", (PyCFunction)(void (*)())py_prompt, METH_FASTCALL, ""},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_rxops", "Marshalling of the row, page and prompt operators.", -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch it was compiled for, whose tensors alone it may read
PyMODINIT_FUNC PyInit__rxops() {
    PyObject* m = PyModule_Create(&module_def);
    if (m && PyModule_AddStringConstant(m, "torch_version", RX_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
