// dg_bind.cpp -- the checks and the marshalling of the serving calls (dg_kv_append, dg_paged_attention,
// dg_adjust_logits) for Python.
//
// These calls are made once a token and a layer, and take 3 to 9 us on the device for a few sequences.
// Checked in Python and passed through ctypes they took the host 10.5 to 12.9 us, which a decoding loop waited
// for; from here 3 us for one kernel and 5 for two, launches included (64 tokens appended one after
// another: 10.6 us a call before, 3.4 now).  The module holds no state but the entry points' addresses, which
// _native.load() gives it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "dg.h"

namespace {

decltype(&dg_kv_append) g_append = nullptr;
decltype(&dg_paged_attention) g_attention = nullptr;
decltype(&dg_paged_attention_workspace_bytes) g_attention_bytes = nullptr;
decltype(&dg_adjust_logits) g_adjust = nullptr;

struct Raised {};   // a Python error is set

[[noreturn]] void refuse(PyObject* kind, const std::string& why) {
    PyErr_SetString(kind, why.c_str());
    throw Raised();
}

std::string type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kDouble: return "torch.float64";
        case at::kInt: return "torch.int32";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

std::string shape_name(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + (s[i] < 0 ? std::string("any") : std::to_string(s[i]));
    return r + ")";
}

// One call's arguments: the first tensor's device is the call's, and the current one.
struct Call {
    const char* fn;
    int64_t dev = 0;
    bool first = true;

    std::string named(const char* name) const { return std::string(fn) + ": " + name; }

    const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type) {
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, named(name) + " must be a tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.scalar_type() != type)
            refuse(PyExc_TypeError, named(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
        if (t.layout() != at::kStrided) refuse(PyExc_TypeError, named(name) + " must be a strided tensor");
        const int64_t d = t.is_cuda() ? t.get_device() : -1;
        if (first) {
            dev = d;
            first = false;
        }
        if (d != dev)
            refuse(PyExc_ValueError, named(name) + " is on " + t.device().str() + ", other tensors of the call on device " +
                                         std::to_string(dev));
        return t;
    }

    // A contiguous tensor of a type and shape (-1: any extent); nullptr for None.
    void* whole(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o, name, type);
        const at::IntArrayRef want(shape.begin(), shape.size());
        bool same = t.dim() == (int64_t)want.size();
        for (size_t i = 0; same && i < want.size(); ++i) same = want[i] < 0 || t.size(i) == want[i];
        if (!same)
            refuse(PyExc_ValueError, named(name) + " must have shape " + shape_name(want) + ", got " + shape_name(t.sizes()));
        if (!t.is_contiguous()) refuse(PyExc_ValueError, named(name) + " must be contiguous");
        return t.data_ptr();
    }

    // t [tokens, heads, d], whose rows hold [heads][d] without gaps: its address and row stride.
    void* rows(PyObject* o, const char* name, int64_t heads, int64_t d, int64_t& tokens, int64_t& ld) {
        const at::Tensor& t = tensor(o, name, at::kBFloat16);
        if (t.dim() != 3 || (heads >= 0 && t.size(1) != heads) || t.size(2) != d)
            refuse(PyExc_ValueError, named(name) + " must have shape " + shape_name({-1, heads, d}) + ", got " +
                                         shape_name(t.sizes()));
        if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != d))
            refuse(PyExc_ValueError, named(name) + "'s heads must follow each other");
        tokens = t.size(0);
        ld = tokens > 1 ? t.stride(0) : t.size(1) * d;
        return t.data_ptr();
    }

    // The raw stream: the caller's, or the current one of the call's device, which must be the current device.
    dg_stream_t stream(PyObject* o) {
        if (dev < 0) refuse(PyExc_ValueError, std::string(fn) + ": device tensors expected");
        const int64_t current = c10::cuda::current_device();
        if (dev != current)
            refuse(PyExc_ValueError, std::string(fn) + ": the tensors are on device " + std::to_string(dev) +
                                         ", the current device is " + std::to_string(current));
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        void* s = PyLong_AsVoidPtr(o);
        if (!s && PyErr_Occurred()) throw Raised();
        return static_cast<dg_stream_t>(s);
    }
};

int64_t integer(PyObject* o, int64_t lo, int64_t hi, const char* fn, const char* name) {
    PyObject* i = PyNumber_Index(o);
    if (!i) throw Raised();
    int over = 0;
    const int64_t v = PyLong_AsLongLongAndOverflow(i, &over);
    Py_DECREF(i);
    if (over || v < lo || v > hi) refuse(PyExc_ValueError, std::string(fn) + ": " + name + " is out of range");
    return v;
}

int64_t int32(PyObject* o, const char* fn, const char* name) { return integer(o, INT32_MIN, INT32_MAX, fn, name); }

// dg_paged_kv of k_cache, v_cache [n_pages, page_size, Hkv, D] (any strides of the first three) and
// page_table [n_seq, max_pages], kv_len [n_seq].
struct Cache {
    dg_paged_kv kv;
    int64_t n_seq, Hkv, D;

    Cache(Call& c, PyObject* ko, PyObject* vo, PyObject* table, PyObject* len) {
        const at::Tensor& k = c.tensor(ko, "k_cache", at::kBFloat16);
        const at::Tensor& v = c.tensor(vo, "v_cache", at::kBFloat16);
        for (const at::Tensor* t : {&k, &v})
            if (t->dim() != 4 || t->stride(3) != 1)
                refuse(PyExc_ValueError, c.named(t == &k ? "k_cache" : "v_cache") +
                                             " must be [n_pages, page_size, Hkv, D] with contiguous heads");
        bool alike = k.sizes() == v.sizes();
        for (int i = 0; alike && i < 3; ++i) alike = k.size(i) == 1 || k.stride(i) == v.stride(i);
        if (!alike) refuse(PyExc_ValueError, std::string(c.fn) + ": k_cache and v_cache must have one layout");
        kv.kv_len = static_cast<const int32_t*>(c.whole(len, "kv_len", at::kInt, {-1}));
        if (len == Py_None) refuse(PyExc_TypeError, c.named("kv_len") + " must be a tensor");
        n_seq = THPVariable_Unpack(len).size(0);
        kv.page_table = static_cast<const int32_t*>(c.whole(table, "page_table", at::kInt, {n_seq, -1}));
        if (table == Py_None) refuse(PyExc_TypeError, c.named("page_table") + " must be a tensor");
        const int64_t max_pages = THPVariable_Unpack(table).size(1);
        Hkv = k.size(2);
        D = k.size(3);
        if (n_seq > INT32_MAX || max_pages > INT32_MAX || k.size(1) > INT32_MAX || Hkv > INT32_MAX || D > INT32_MAX)
            refuse(PyExc_ValueError, std::string(c.fn) + ": an extent of the cache is out of range");
        kv.k = static_cast<uint16_t*>(k.data_ptr());
        kv.v = static_cast<uint16_t*>(v.data_ptr());
        kv.n_pages = k.size(0);
        // the stride of an extent of one says nothing: any valid one will do
        kv.page_stride = k.size(0) > 1 ? k.stride(0) : D;
        kv.slot_stride = k.size(1) > 1 ? k.stride(1) : D;
        kv.head_stride = k.size(2) > 1 ? k.stride(2) : D;
        kv.page_size = (int32_t)k.size(1);
        kv.max_pages = (int32_t)max_pages;
    }
};

template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool takes(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}

// k, v, k_cache, v_cache, page_table, cu_q, kv_len, inv_freq, interleaved, q, q_out, stream -> status
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!takes(n, 12)) return nullptr;
    return guarded([&]() -> PyObject* {
        Call c{"dg_kv_append"};
        PyObject *q = a[9], *q_out = a[10];
        if ((q == Py_None) != (q_out == Py_None)) refuse(PyExc_ValueError, "dg_kv_append: q and q_out come together");
        const Cache kv(c, a[2], a[3], a[4], a[6]);
        int64_t total, ldk, v_rows, ldv, q_rows = 0, ldq = 0, Hq = kv.Hkv;
        const void* kp = c.rows(a[0], "k", kv.Hkv, kv.D, total, ldk);
        const void* vp = c.rows(a[1], "v", kv.Hkv, kv.D, v_rows, ldv);
        const void* qp = nullptr;
        void* op = nullptr;
        if (q != Py_None) {
            qp = c.rows(q, "q", -1, kv.D, q_rows, ldq);
            Hq = THPVariable_Unpack(q).size(1);
            op = c.whole(q_out, "q_out", at::kBFloat16, {q_rows, Hq, kv.D});
        }
        if (v_rows != total || (q != Py_None && q_rows != total))
            refuse(PyExc_ValueError, "dg_kv_append: q, k and v must have as many rows");
        if (Hq > INT32_MAX) refuse(PyExc_ValueError, "dg_kv_append: too many heads");
        const void* cu = c.whole(a[5], "cu_q", at::kInt, {kv.n_seq + 1});
        const void* w = c.whole(a[7], "inv_freq", at::kDouble, {-1});
        const int64_t half = w || a[7] != Py_None ? THPVariable_Unpack(a[7]).size(0) : 0;
        if (half > INT32_MAX / 2) refuse(PyExc_ValueError, "dg_kv_append: inv_freq is too long");
        const int interleaved = PyObject_IsTrue(a[8]);
        if (interleaved < 0) throw Raised();
        const dg_stream_t st = c.stream(a[11]);
        dg_status rc;
        Py_BEGIN_ALLOW_THREADS;
        rc = g_append((const uint16_t*)kp, ldk, (const uint16_t*)vp, ldv, (const uint16_t*)qp, ldq, (uint16_t*)op,
                      (const int32_t*)cu, (int32_t)kv.n_seq, total, (int32_t)Hq, (int32_t)kv.Hkv, (int32_t)kv.D,
                      (const double*)w, (int32_t)(2 * half), interleaved, &kv.kv, st);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(rc);
    });
}

// q, k_cache, v_cache, o, page_table, cu_q, kv_len, causal, max_q_len, lse, window, scale, workspace, stream
// -> status; without a workspace nothing runs, and the bytes it needs come back as a 1-tuple
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!takes(n, 14)) return nullptr;
    return guarded([&]() -> PyObject* {
        const char* fn = "dg_paged_attention";
        Call c{fn};
        const Cache kv(c, a[1], a[2], a[4], a[6]);
        const void* q = c.whole(a[0], "q", at::kBFloat16, {-1, -1, kv.D});
        if (a[0] == Py_None) refuse(PyExc_TypeError, c.named("q") + " must be a tensor");
        const at::Tensor& qt = THPVariable_Unpack(a[0]);
        const int64_t total = qt.size(0), Hq = qt.size(1);
        if (Hq > INT32_MAX) refuse(PyExc_ValueError, c.named("q") + " has too many heads");
        void* o = c.whole(a[3], "o", at::kBFloat16, {total, Hq, kv.D});
        const void* cu = c.whole(a[5], "cu_q", at::kInt, {kv.n_seq + 1});
        const void* causal = c.whole(a[7], "causal", at::kByte, {kv.n_seq});
        void* lse = c.whole(a[9], "lse", at::kFloat, {total, Hq});
        const int64_t max_q = int32(a[8], fn, "max_q_len"), window = int32(a[10], fn, "window");
        double scale = kv.D > 0 ? 1.0 / std::sqrt((double)kv.D) : 0.0;
        if (a[11] != Py_None) {
            scale = PyFloat_AsDouble(a[11]);
            if (scale == -1.0 && PyErr_Occurred()) throw Raised();
        }
        const dg_stream_t st = c.stream(a[13]);
        if (a[12] == Py_None)
            return Py_BuildValue("(n)", (Py_ssize_t)g_attention_bytes((int32_t)kv.n_seq, (int32_t)max_q, (int32_t)Hq,
                                                                      (int32_t)kv.Hkv, (int32_t)kv.D));
        if (!THPVariable_Check(a[12])) refuse(PyExc_TypeError, c.named("workspace") + " must be a tensor");
        const at::Tensor& ws = c.tensor(a[12], "workspace", THPVariable_Unpack(a[12]).scalar_type());
        if (!ws.is_contiguous()) refuse(PyExc_ValueError, c.named("workspace") + " must be contiguous");
        void* wp = ws.data_ptr();
        const size_t bytes = ws.nbytes();
        dg_status rc;
        Py_BEGIN_ALLOW_THREADS;
        rc = g_attention((const uint16_t*)q, &kv.kv, (uint16_t*)o, (float*)lse, (const int32_t*)cu, (const uint8_t*)causal,
                         (int32_t)kv.n_seq, (int32_t)max_q, total, (int32_t)Hq, (int32_t)kv.Hkv, (int32_t)kv.D,
                         (int32_t)window, (float)scale, wp, bytes, st);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(rc);
    });
}

// logits, params, out, history, cu_history, penalties, bias_tokens, bias_values, cu_bias, masks, mask_index, V,
// stream, bytes of a canvas's params -> status
PyObject* adjust_logits(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!takes(n_args, 14)) return nullptr;
    return guarded([&]() -> PyObject* {
        const char* fn = "dg_adjust_logits";
        Call c{fn};
        PyObject *logits = a[0], *out = a[2] == Py_None ? a[0] : a[2];
        if (!THPVariable_Check(logits)) refuse(PyExc_TypeError, c.named("logits") + " must be a tensor");
        const at::ScalarType type = THPVariable_Unpack(logits).scalar_type();
        if (type != at::kBFloat16 && type != at::kFloat) refuse(PyExc_TypeError, "logits must be bfloat16 or float32");
        void* x = c.whole(logits, "logits", type, {-1, -1, -1});
        const at::Tensor& xt = THPVariable_Unpack(logits);
        const int64_t n = xt.size(0), L = xt.size(1), ld = xt.size(2);
        void* o = c.whole(out, "out", type, {n, L, -1});
        const int64_t ldo = THPVariable_Unpack(out).size(2);
        const int64_t V = a[11] == Py_None ? ld : integer(a[11], INT64_MIN, INT64_MAX, fn, "V");
        auto together = [&](std::initializer_list<int> at, const char* names) {
            for (int i : at)
                if ((a[i] == Py_None) != (a[*at.begin()] == Py_None))
                    refuse(PyExc_ValueError, std::string(fn) + ": " + names + " come together");
        };
        together({3, 4, 5}, "history, cu_history and penalties");
        together({6, 7, 8}, "bias_tokens, bias_values and cu_bias");
        together({9, 10}, "masks and mask_index");
        const void* p = c.whole(a[1], "params", at::kByte, {n * integer(a[13], 0, 1 << 20, fn, "params")});
        if (a[1] == Py_None) refuse(PyExc_TypeError, c.named("params") + " must be a tensor");
        const void* h = c.whole(a[3], "history", at::kInt, {-1});
        const int64_t nh = a[3] == Py_None ? 0 : THPVariable_Unpack(a[3]).size(0);
        const void* ch = c.whole(a[4], "cu_history", at::kInt, {n + 1});
        const void* pen = c.whole(a[5], "penalties", at::kFloat, {n, 3});
        const void* bt = c.whole(a[6], "bias_tokens", at::kInt, {-1});
        const int64_t nb = a[6] == Py_None ? 0 : THPVariable_Unpack(a[6]).size(0);
        const void* bv = c.whole(a[7], "bias_values", at::kFloat, {nb});
        const void* cb = c.whole(a[8], "cu_bias", at::kInt, {n + 1});
        const void* m = c.whole(a[9], "masks", at::kInt, {-1, -1});
        int64_t n_masks = 0, words = 0;
        if (a[9] != Py_None) {
            n_masks = THPVariable_Unpack(a[9]).size(0);
            words = THPVariable_Unpack(a[9]).size(1);
            if (n_masks < 1 || words < 1) refuse(PyExc_ValueError, c.named("masks") + " must have rows and words");
        }
        const void* mi = c.whole(a[10], "mask_index", at::kInt, {n, L});
        if (L > INT32_MAX || n_masks > INT32_MAX) refuse(PyExc_ValueError, std::string(fn) + ": an extent is out of range");
        const dg_stream_t st = c.stream(a[12]);
        dg_status rc;
        Py_BEGIN_ALLOW_THREADS;
        rc = g_adjust(x, type == at::kBFloat16 ? DG_BF16 : DG_FP32, ld, o, ldo, n, (int32_t)L, V, (const dg_canvas_params*)p,
                      (const int32_t*)h, (const int32_t*)ch, nh, (const dg_penalties*)pen, (const int32_t*)bt,
                      (const float*)bv, (const int32_t*)cb, nb, (const uint32_t*)m, words, (int32_t)n_masks,
                      (const int32_t*)mi, st);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(rc);
    });
}

// The addresses of dg_kv_append, dg_paged_attention, its workspace query and dg_adjust_logits.
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!takes(n, 4)) return nullptr;
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
            return nullptr;
        }
    }
    g_append = reinterpret_cast<decltype(g_append)>(p[0]);
    g_attention = reinterpret_cast<decltype(g_attention)>(p[1]);
    g_attention_bytes = reinterpret_cast<decltype(g_attention_bytes)>(p[2]);
    g_adjust = reinterpret_cast<decltype(g_adjust)>(p[3]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef kMethods[] = {{"connect", fast<connect>(), METH_FASTCALL, nullptr},
                          {"kv_append", fast<kv_append>(), METH_FASTCALL, nullptr},
                          {"paged_attention", fast<paged_attention>(), METH_FASTCALL, nullptr},
                          {"adjust_logits", fast<adjust_logits>(), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "dg_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_dg_bind() { return PyModule_Create(&kModule); }
