// dg_bind.cpp -- the checks and the marshalling of the serving calls (dg_kv_append, dg_paged_attention,
// dg_adjust_logits, and for drafted tokens dg_kv_append_norm, dg_tree_attention, dg_sink_attention,
// dg_verify_drafts, dg_kv_keep) for Python.
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
decltype(&dg_kv_append_norm) g_append_norm = nullptr;
decltype(&dg_tree_attention) g_tree = nullptr;
decltype(&dg_tree_attention_workspace_bytes) g_tree_bytes = nullptr;
decltype(&dg_sink_attention) g_sink = nullptr;
decltype(&dg_verify_drafts) g_verify = nullptr;
decltype(&dg_kv_keep) g_keep = nullptr;

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
// page_table [n_seq, max_pages], kv_len [n_seq]; where `layers` allows it, of [n_layers, n_pages, ...] too.
struct Cache {
    dg_paged_kv kv;
    int64_t n_seq, Hkv, D, n_layers = 1, layer_stride = 0;

    Cache(Call& c, PyObject* ko, PyObject* vo, PyObject* table, PyObject* len, bool layers = false) {
        const at::Tensor& kt = c.tensor(ko, "k_cache", at::kBFloat16);
        const at::Tensor& vt = c.tensor(vo, "v_cache", at::kBFloat16);
        for (const at::Tensor* t : {&kt, &vt})
            if ((t->dim() != 4 && !(layers && t->dim() == 5)) || t->stride(t->dim() - 1) != 1)
                refuse(PyExc_ValueError, c.named(t == &kt ? "k_cache" : "v_cache") + " must be [" +
                                             (layers ? "n_layers (or not), " : "") +
                                             "n_pages, page_size, Hkv, D] with contiguous heads");
        const int skip = kt.dim() == 5 ? 1 : 0;
        struct View {   // the four extents and strides of a layer
            const at::Tensor& t;
            int skip;
            int64_t size(int i) const { return t.size(i + skip); }
            int64_t stride(int i) const { return t.stride(i + skip); }
            void* data_ptr() const { return t.data_ptr(); }
        };
        const View k{kt, skip}, v{vt, skip};
        bool alike = kt.sizes() == vt.sizes();
        for (int i = 0; alike && i < 3; ++i) alike = k.size(i) == 1 || k.stride(i) == v.stride(i);
        if (alike && skip) {
            n_layers = kt.size(0);
            layer_stride = n_layers > 1 ? kt.stride(0) : 0;
            alike = n_layers <= 1 || kt.stride(0) == vt.stride(0);
            if (n_layers > INT32_MAX) refuse(PyExc_ValueError, std::string(c.fn) + ": an extent of the cache is out of range");
        }
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

// k, v, k_cache, v_cache, page_table, cu_q, kv_len, inv_freq, interleaved, q, q_out, stream -> status;
// with norms q_norm, k_norm, eps, positions follow
template <bool Norm>
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!takes(n, Norm ? 16 : 12)) return nullptr;
    return guarded([&]() -> PyObject* {
        const std::string fn = Norm ? "dg_kv_append_norm" : "dg_kv_append";
        Call c{fn.c_str()};
        PyObject *q = a[9], *q_out = a[10];
        if ((q == Py_None) != (q_out == Py_None)) refuse(PyExc_ValueError, fn + ": q and q_out come together");
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
            refuse(PyExc_ValueError, fn + ": q, k and v must have as many rows");
        if (Hq > INT32_MAX) refuse(PyExc_ValueError, fn + ": too many heads");
        const void* cu = c.whole(a[5], "cu_q", at::kInt, {kv.n_seq + 1});
        const void* w = c.whole(a[7], "inv_freq", at::kDouble, {-1});
        const int64_t half = w || a[7] != Py_None ? THPVariable_Unpack(a[7]).size(0) : 0;
        if (half > INT32_MAX / 2) refuse(PyExc_ValueError, fn + ": inv_freq is too long");
        const int interleaved = PyObject_IsTrue(a[8]);
        if (interleaved < 0) throw Raised();
        const void *qn = nullptr, *kn = nullptr, *pos = nullptr;
        double eps = 0.0;
        if constexpr (Norm) {
            qn = c.whole(a[12], "q_norm", at::kFloat, {kv.D});
            kn = c.whole(a[13], "k_norm", at::kFloat, {kv.D});
            if (a[12] != Py_None && q == Py_None) refuse(PyExc_ValueError, fn + ": q_norm comes with q");
            eps = PyFloat_AsDouble(a[14]);
            if (eps == -1.0 && PyErr_Occurred()) throw Raised();
            pos = c.whole(a[15], "positions", at::kInt, {total});
        }
        const dg_stream_t st = c.stream(a[11]);
        dg_status rc;
        Py_BEGIN_ALLOW_THREADS;
        if constexpr (Norm)
            rc = g_append_norm((const uint16_t*)kp, ldk, (const uint16_t*)vp, ldv, (const uint16_t*)qp, ldq, (uint16_t*)op,
                               (const int32_t*)cu, (int32_t)kv.n_seq, total, (int32_t)Hq, (int32_t)kv.Hkv, (int32_t)kv.D,
                               (const float*)qn, (const float*)kn, (float)eps, (const int32_t*)pos, (const double*)w,
                               (int32_t)(2 * half), interleaved, &kv.kv, st);
        else
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

// q, k_cache, v_cache, o, page_table, cu_q, kv_len, max_q_len, lse, window, sinks, scale, workspace, stream and, of a tree,
// tree_mask, positions -> status; without a workspace nothing runs, and the bytes it needs come back as a 1-tuple
template <bool Tree>
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!takes(n, Tree ? 16 : 14)) return nullptr;
    return guarded([&]() -> PyObject* {
        const char* fn = Tree ? "dg_tree_attention" : "dg_sink_attention";
        Call c{fn};
        const Cache kv(c, a[1], a[2], a[4], a[6]);
        const void* q = c.whole(a[0], "q", at::kBFloat16, {-1, -1, kv.D});
        if (a[0] == Py_None) refuse(PyExc_TypeError, c.named("q") + " must be a tensor");
        const at::Tensor& qt = THPVariable_Unpack(a[0]);
        const int64_t total = qt.size(0), Hq = qt.size(1);
        if (Hq > INT32_MAX) refuse(PyExc_ValueError, c.named("q") + " has too many heads");
        void* o = c.whole(a[3], "o", at::kBFloat16, {total, Hq, kv.D});
        const void* cu = c.whole(a[5], "cu_q", at::kInt, {kv.n_seq + 1});
        void* lse = c.whole(a[8], "lse", at::kFloat, {total, Hq});
        const int64_t max_q = int32(a[7], fn, "max_q_len"), window = int32(a[9], fn, "window"), sinks = int32(a[10], fn, "sinks");
        double scale = kv.D > 0 ? 1.0 / std::sqrt((double)kv.D) : 0.0;
        if (a[11] != Py_None) {
            scale = PyFloat_AsDouble(a[11]);
            if (scale == -1.0 && PyErr_Occurred()) throw Raised();
        }
        const void *mask = nullptr, *pos = nullptr;
        int64_t words = 0;
        if constexpr (Tree) {
            mask = c.whole(a[14], "tree_mask", at::kInt, {total, -1});
            if (a[14] == Py_None) refuse(PyExc_TypeError, c.named("tree_mask") + " must be a tensor");
            words = THPVariable_Unpack(a[14]).size(1);
            if (words > INT32_MAX) refuse(PyExc_ValueError, c.named("tree_mask") + " has too many words");
            pos = c.whole(a[15], "positions", at::kInt, {total});
        }
        const dg_stream_t st = c.stream(a[13]);
        if (a[12] == Py_None)
            return Py_BuildValue("(n)", (Py_ssize_t)g_tree_bytes((int32_t)kv.n_seq, (int32_t)max_q, (int32_t)Hq,
                                                                 (int32_t)kv.Hkv, (int32_t)kv.D));
        if (!THPVariable_Check(a[12])) refuse(PyExc_TypeError, c.named("workspace") + " must be a tensor");
        const at::Tensor& ws = c.tensor(a[12], "workspace", THPVariable_Unpack(a[12]).scalar_type());
        if (!ws.is_contiguous()) refuse(PyExc_ValueError, c.named("workspace") + " must be contiguous");
        void* wp = ws.data_ptr();
        const size_t bytes = ws.nbytes();
        dg_status rc;
        Py_BEGIN_ALLOW_THREADS;
        if constexpr (Tree)
            rc = g_tree((const uint16_t*)q, &kv.kv, (uint16_t*)o, (float*)lse, (const int32_t*)cu, (const uint32_t*)mask,
                        (int32_t)words, (const int32_t*)pos, (int32_t)kv.n_seq, (int32_t)max_q, total, (int32_t)Hq,
                        (int32_t)kv.Hkv, (int32_t)kv.D, (int32_t)window, (int32_t)sinks, (float)scale, wp, bytes, st);
        else
            rc = g_sink((const uint16_t*)q, &kv.kv, (uint16_t*)o, (float*)lse, (const int32_t*)cu, (int32_t)kv.n_seq,
                        (int32_t)max_q, total, (int32_t)Hq, (int32_t)kv.Hkv, (int32_t)kv.D, (int32_t)window,
                        (int32_t)sinks, (float)scale, wp, bytes, st);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(rc);
    });
}

// logits, tokens, cu_q, temperature, uniforms, next_uniforms, n_accept, path, out_tokens, parents, draft_probs, V, stream
// -> status
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!takes(n_args, 13)) return nullptr;
    return guarded([&]() -> PyObject* {
        const char* fn = "dg_verify_drafts";
        Call c{fn};
        if (!THPVariable_Check(a[0])) refuse(PyExc_TypeError, c.named("logits") + " must be a tensor");
        const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
        if (type != at::kBFloat16 && type != at::kFloat) refuse(PyExc_TypeError, "logits must be bfloat16 or float32");
        // rows of any stride: the last dimension's elements follow each other.  A single row's stride says how far apart the
        // rows of its buffer lie, and counts where the library needs more columns than the row has and they lie there.
        auto rows = [&](PyObject* o, const char* name, at::ScalarType t, int64_t& ld) -> const at::Tensor& {
            const at::Tensor& x = c.tensor(o, name, t);
            if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1))
                refuse(PyExc_ValueError, c.named(name) + " must be [total, columns] with contiguous rows");
            ld = x.size(0) > 1 ? x.stride(0) : x.size(1);
            const int64_t es = (int64_t)x.element_size(), held = (int64_t)x.storage().nbytes() / es - x.storage_offset();
            if (x.size(0) == 1 && ld * es % 16 && x.stride(0) > ld && (ld * es + 15) / 16 * 16 <= held * es) ld = x.stride(0);
            return x;
        };
        int64_t ld, ldq = 0;
        const at::Tensor& x = rows(a[0], "logits", type, ld);
        const int64_t total = x.size(0), V = a[11] == Py_None ? x.size(1) : integer(a[11], INT64_MIN, INT64_MAX, fn, "V");
        if (V > x.size(1)) refuse(PyExc_ValueError, c.named("V") + " is more than the logits' columns");
        for (int i : {1, 2, 3, 4, 5, 6, 7, 8})
            if (a[i] == Py_None) refuse(PyExc_TypeError, std::string(fn) + ": an argument is None");
        c.whole(a[3], "temperature", at::kFloat, {-1});
        const int64_t n = THPVariable_Unpack(a[3]).size(0);
        if (n > INT32_MAX) refuse(PyExc_ValueError, std::string(fn) + ": too many sequences");
        const void* temperature = c.whole(a[3], "temperature", at::kFloat, {n});
        const void* tokens = c.whole(a[1], "tokens", at::kInt, {total});
        const void* cu = c.whole(a[2], "cu_q", at::kInt, {n + 1});
        const void* u = c.whole(a[4], "uniforms", at::kFloat, {total});
        const void* un = c.whole(a[5], "next_uniforms", at::kFloat, {n});
        void* count = c.whole(a[6], "n_accept", at::kInt, {n});
        void* path = c.whole(a[7], "path", at::kInt, {total});
        void* out = c.whole(a[8], "out_tokens", at::kInt, {total});
        const void* parents = c.whole(a[9], "parents", at::kInt, {total});
        const void* probs = nullptr;
        if (a[10] != Py_None) {
            const at::Tensor& p = rows(a[10], "draft_probs", at::kFloat, ldq);
            if (p.size(0) != total || p.size(1) < V)
                refuse(PyExc_ValueError, c.named("draft_probs") + " must have the logits' rows and at least V columns");
            if (a[9] != Py_None) refuse(PyExc_ValueError, std::string(fn) + ": parents and draft_probs do not go together");
            probs = p.data_ptr();
        }
        const dg_stream_t st = c.stream(a[12]);
        dg_status rc;
        Py_BEGIN_ALLOW_THREADS;
        rc = g_verify(x.data_ptr(), type == at::kBFloat16 ? DG_BF16 : DG_FP32, ld, (const int32_t*)tokens,
                      (const int32_t*)parents, (const float*)probs, ldq, (const int32_t*)cu, (int32_t)n, total, V,
                      (const float*)temperature, (const float*)u, (const float*)un, (int32_t*)count, (int32_t*)path,
                      (int32_t*)out, st);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(rc);
    });
}

// k_cache, v_cache, page_table, cu_q, kv_len, path, n_accept, new_len, stream -> status
PyObject* kv_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!takes(n, 9)) return nullptr;
    return guarded([&]() -> PyObject* {
        Call c{"dg_kv_keep"};
        const Cache kv(c, a[0], a[1], a[2], a[4], true);
        for (int i : {3, 5, 6, 7})
            if (a[i] == Py_None) refuse(PyExc_TypeError, std::string(c.fn) + ": an argument is None");
        const void* cu = c.whole(a[3], "cu_q", at::kInt, {kv.n_seq + 1});
        const void* path = c.whole(a[5], "path", at::kInt, {-1});
        const int64_t total = THPVariable_Unpack(a[5]).size(0);
        const void* count = c.whole(a[6], "n_accept", at::kInt, {kv.n_seq});
        void* len = c.whole(a[7], "new_len", at::kInt, {kv.n_seq});
        const dg_stream_t st = c.stream(a[8]);
        dg_status rc;
        Py_BEGIN_ALLOW_THREADS;
        rc = g_keep(&kv.kv, (int32_t)kv.n_layers, kv.layer_stride, (const int32_t*)cu, (int32_t)kv.n_seq, total,
                    (int32_t)kv.Hkv, (int32_t)kv.D, (const int32_t*)path, (const int32_t*)count, (int32_t*)len, st);
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

// The addresses of dg_kv_append, dg_paged_attention, its workspace query, dg_adjust_logits, dg_kv_append_norm,
// dg_tree_attention, its workspace query, dg_sink_attention, dg_verify_drafts and dg_kv_keep.
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
    constexpr int kCalls = 10;
    if (!takes(n, kCalls)) return nullptr;
    void* p[kCalls];
    for (int i = 0; i < kCalls; ++i) {
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
    g_append_norm = reinterpret_cast<decltype(g_append_norm)>(p[4]);
    g_tree = reinterpret_cast<decltype(g_tree)>(p[5]);
    g_tree_bytes = reinterpret_cast<decltype(g_tree_bytes)>(p[6]);
    g_sink = reinterpret_cast<decltype(g_sink)>(p[7]);
    g_verify = reinterpret_cast<decltype(g_verify)>(p[8]);
    g_keep = reinterpret_cast<decltype(g_keep)>(p[9]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef kMethods[] = {{"connect", fast<connect>(), METH_FASTCALL, nullptr},
                          {"kv_append", fast<kv_append<false>>(), METH_FASTCALL, nullptr},
                          {"kv_append_norm", fast<kv_append<true>>(), METH_FASTCALL, nullptr},
                          {"tree_attention", fast<tree_attention<true>>(), METH_FASTCALL, nullptr},
                          {"sink_attention", fast<tree_attention<false>>(), METH_FASTCALL, nullptr},
                          {"verify_drafts", fast<verify_drafts>(), METH_FASTCALL, nullptr},
                          {"kv_keep", fast<kv_keep>(), METH_FASTCALL, nullptr},
                          {"paged_attention", fast<paged_attention>(), METH_FASTCALL, nullptr},
                          {"adjust_logits", fast<adjust_logits>(), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "dg_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_dg_bind() { return PyModule_Create(&kModule); }
