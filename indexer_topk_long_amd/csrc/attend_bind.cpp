// attend_bind.cpp -- Python entry of the paged cache's operators.
//
// A decode step's calls take a few microseconds on the GPU, as long as reading
// ten tensors' attributes from Python takes.  This module does that reading,
// the checks and the launches: every function takes positional arguments in
// the order of its wrapper in attention.py, which documents them.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <math.h>

#include <string>

#include "litetopk_attend.h"

namespace {

// Thrown after a Python error has been set.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const std::string& msg) {
    PyErr_SetString(type, msg.c_str());
    throw Refused{};
}

[[noreturn]] void failed(int status, const char* where) {
    PyObject* mod = PyImport_ImportModule("indexer_topk_long_amd._binding");
    PyObject* cls = mod ? PyObject_GetAttrString(mod, "LtkError") : nullptr;
    PyObject* err = cls ? PyObject_CallFunction(cls, "is", status, where) : nullptr;
    if (err) PyErr_SetObject(cls, err);
    Py_XDECREF(err);
    Py_XDECREF(cls);
    Py_XDECREF(mod);
    throw Refused{};
}

std::string shape_text(c10::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

struct Kind {
    at::ScalarType type;
    const char* name;
};
constexpr Kind kBf16{at::kBFloat16, "torch.bfloat16"}, kFp8{at::kFloat8_e4m3fn, "torch.float8_e4m3fn"},
    kF32{at::kFloat, "torch.float32"}, kF64{at::kDouble, "torch.float64"}, kI32{at::kInt, "torch.int32"},
    kU32{at::kUInt32, "torch.uint32"};

// The operators compute no gradients: a result would silently be detached from
// a tensor that autograd follows, backward or forward.
void without_grad(const at::Tensor& t, const char* name) {
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse(PyExc_RuntimeError, std::string(name) + " requires grad: the paged cache's operators are forward only "
                                                       "(call them under torch.no_grad(), or detach it)");
    if (t.unsafeGetTensorImpl()->_fw_grad(0, t).defined())   // (read in place: as an operator it goes through the dispatcher)
        refuse(PyExc_RuntimeError, std::string(name) + " carries a tangent: the paged cache's operators are forward only");
}

// After a call has written a tensor in place: autograd sees that what it saved
// of it has changed.  (Inference tensors count no versions.)
void in_place(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A contiguous device tensor of this type and shape (-1: any size), on the
// cache's device where dev >= 0.
const at::Tensor& tensor(PyObject* o, const char* name, Kind kind, std::initializer_list<int64_t> want, int dev) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != kind.type)
        refuse(PyExc_TypeError, std::string(name) + " must be " + kind.name + ", got " + c10::toString(t.scalar_type()));
    const auto got = t.sizes();
    bool ok = got.size() == want.size();
    for (size_t i = 0; ok && i < got.size(); ++i) ok = want.begin()[i] < 0 || want.begin()[i] == got[i];
    if (!ok) {
        std::string w;
        for (int64_t n : want) w += (w.empty() ? "" : ", ") + (n < 0 ? std::string("*") : std::to_string(n));
        refuse(PyExc_ValueError, std::string(name) + " must be [" + w + "], got " + shape_text(got));
    }
    without_grad(t, name);
    if (!t.is_cuda() || !t.is_contiguous())
        refuse(PyExc_ValueError, std::string(name) + " must be a contiguous device tensor");
    if (dev >= 0 && t.get_device() != dev)
        refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the cache on cuda:" +
                                     std::to_string(dev) + ": all tensors must share one device");
    return t;
}

int int32_of(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
    return (int)v;
}

int32_t size32(int64_t n, const char* name) {
    if (n > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is too large");
    return (int32_t)n;
}

struct Cache {
    ltk_kv_cache c;
    int dev;
    at::Tensor tensors[4];   // held: reading a later argument may run Python code that takes them from a list
    void written() const {
        for (const at::Tensor& t : tensors) in_place(t);
    }
};
Cache cache_of(PyObject* o) {
    PyObject** e = PyTuple_Check(o) ? &PyTuple_GET_ITEM(o, 0) : nullptr;
    Py_ssize_t n = e ? PyTuple_GET_SIZE(o) : 0;
    if (PyList_Check(o)) n = PyList_GET_SIZE(o), e = n ? &PyList_GET_ITEM(o, 0) : nullptr;
    if (n != 4) refuse(PyExc_ValueError, "cache must be (k, v, k_scale, v_scale)");
    const at::Tensor& k = tensor(e[0], "cache k", kFp8, {-1, -1, -1, -1}, -1);
    const int dev = k.get_device();
    const auto s = k.sizes();
    Cache r;
    r.dev = dev;
    r.c.k = k.data_ptr();
    r.c.v = tensor(e[1], "cache v", kFp8, {s[0], s[1], s[2], s[3]}, dev).data_ptr();
    r.c.k_scale = static_cast<float*>(tensor(e[2], "k_scale", kF32, {s[0], s[1]}, dev).data_ptr());
    r.c.v_scale = static_cast<float*>(tensor(e[3], "v_scale", kF32, {s[0], s[1]}, dev).data_ptr());
    for (int i = 0; i < 4; ++i) r.tensors[i] = THPVariable_Unpack(e[i]);
    r.c.n_pages = size32(s[0], "the cache");
    r.c.n_kv_heads = size32(s[1], "the cache");
    r.c.page_size = size32(s[2], "the cache");
    r.c.head_dim = size32(s[3], "the cache");
    return r;
}

// cu == NULL: the packed kind, which has none.
ltk_kv_batch batch_of(PyObject* page_table, PyObject* cu, PyObject* kv_len, int dev) {
    const at::Tensor& pt = tensor(page_table, "page_table", kI32, {-1, -1}, dev);
    ltk_kv_batch b;
    b.n_seq = size32(pt.size(0), "page_table");
    b.max_pages = size32(pt.size(1), "page_table");
    b.page_table = static_cast<const int32_t*>(pt.data_ptr());
    b.cu = cu ? static_cast<const int32_t*>(tensor(cu, "cu", kI32, {(int64_t)b.n_seq + 1}, dev).data_ptr()) : nullptr;
    b.kv_len = static_cast<const int32_t*>(tensor(kv_len, "kv_len", kI32, {b.n_seq}, dev).data_ptr());
    return b;
}

// The library launches on the current device: makes the cache's current.
struct On {
    c10::DeviceIndex was;
    int dev;
    void* stream;
    explicit On(int d) : was(c10::hip::current_device()), dev(d) {
        if (was != dev) c10::hip::set_device((c10::DeviceIndex)dev);
        stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
    }
    ~On() {
        if (was != dev) {
            try {
                c10::hip::set_device(was);
            } catch (...) {
            }
        }
    }
    On(const On&) = delete;
    On& operator=(const On&) = delete;
};

at::TensorOptions on_device(int dev, at::ScalarType t) {
    return at::TensorOptions().dtype(t).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
}

// What every attend call starts from: queries, output, workspace.
struct Call {
    Cache cache;
    ltk_kv_batch batch;
    const void* q;
    int32_t T, Hq;
    float scale;
    at::Tensor out, ws;
    bool own_out;
    size_t ws_bytes;
    void* ws_at;

    Call(PyObject* cache_o, PyObject* pt, PyObject* cu, PyObject* len, PyObject* q_o, PyObject* scale_o, PyObject* out_o)
        : cache(cache_of(cache_o)), batch(batch_of(pt, cu, len, cache.dev)) {
        const ltk_kv_cache& c = cache.c;
        const at::Tensor& qt = tensor(q_o, "q", kBf16, {-1, -1, c.head_dim}, cache.dev);
        T = size32(qt.size(0), "q");
        Hq = size32(qt.size(1), "q");
        if (Hq < 1 || Hq % (c.n_kv_heads > 0 ? c.n_kv_heads : 1) != 0)
            refuse(PyExc_ValueError, "q has " + std::to_string(Hq) + " heads, the cache " + std::to_string(c.n_kv_heads) +
                                         ": not a multiple");
        q = qt.data_ptr();
        scale = 1.0f / sqrtf((float)c.head_dim);
        if (scale_o != Py_None) {
            const double s = PyFloat_AsDouble(scale_o);
            if (s == -1.0 && PyErr_Occurred()) throw Refused{};
            scale = (float)s;
        }
        own_out = out_o == Py_None;
        out = own_out ? at::empty({T, Hq, c.head_dim}, on_device(cache.dev, at::kBFloat16))
                      : tensor(out_o, "out", kBf16, {T, Hq, c.head_dim}, cache.dev);
    }

    void workspace(int kind, int64_t entries, int group, PyObject* o) {
        const ltk_kv_cache& c = cache.c;
        if (o == Py_None) {
            const size_t need =
                litetopk_attend_workspace_bytes(kind, T, Hq, c.n_kv_heads, c.head_dim, batch.n_seq, entries, group);
            // (sizes the library does not take: it says so itself, before it looks at the workspace)
            ws_bytes = need ? need : 256;
            ws = at::empty({(int64_t)ws_bytes}, on_device(cache.dev, at::kByte));
        } else {
            if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "workspace must be a tensor");
            ws = THPVariable_Unpack(o);
            ws_bytes = (size_t)ws.numel() * ws.element_size();
            if (!ws.is_cuda() || !ws.is_contiguous() || ws.get_device() != cache.dev)
                refuse(PyExc_ValueError, "workspace must be a contiguous tensor on the cache's device");
        }
        ws_at = ws.data_ptr();
    }

    PyObject* result(int rc, const char* where, PyObject* out_o) {
        if (rc == LTK_EWORKSPACE)
            refuse(PyExc_ValueError, "workspace too small: " + std::to_string(ws_bytes) +
                                         " bytes (attend_workspace_bytes gives what suffices)");
        if (rc != LTK_OK) failed(rc, where);
        if (own_out) return THPVariable_Wrap(out);
        in_place(out);
        Py_INCREF(out_o);
        return out_o;
    }
};

void expect_args(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse(PyExc_TypeError, "expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

template <class F>
PyObject* guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 10);
        PyObject *k_o = a[0], *v_o = a[1], *f_o = a[6], *q_o = a[7], *qo_o = a[9];
        const Cache cache = cache_of(a[2]);
        const ltk_kv_cache& c = cache.c;
        const ltk_kv_batch b = batch_of(a[3], a[4], a[5], cache.dev);
        const at::Tensor& k = tensor(k_o, "k", kBf16, {-1, c.n_kv_heads, c.head_dim}, cache.dev);
        const int32_t T = size32(k.size(0), "k");
        const at::Tensor& v = tensor(v_o, "v", kBf16, {T, c.n_kv_heads, c.head_dim}, cache.dev);
        const double* f = nullptr;
        int32_t rot = 0, Hq = 0;
        if (f_o != Py_None) {
            const at::Tensor& t = tensor(f_o, "inv_freq", kF64, {-1}, cache.dev);
            f = static_cast<const double*>(t.data_ptr());
            rot = size32(2 * t.size(0), "inv_freq");
        }
        const void* q = nullptr;
        void* q_out = nullptr;
        at::Tensor qo;
        if (q_o != Py_None) {
            const at::Tensor& t = tensor(q_o, "q", kBf16, {T, -1, c.head_dim}, cache.dev);
            q = t.data_ptr();
            Hq = size32(t.size(1), "q");
            qo = qo_o == Py_None ? at::empty({T, Hq, c.head_dim}, on_device(cache.dev, at::kBFloat16))
                                 : tensor(qo_o, "q_out", kBf16, {T, Hq, c.head_dim}, cache.dev);
            q_out = qo.data_ptr();
            if (T == 0) q = q_out = nullptr;   // (an empty tensor may have no address)
        } else if (qo_o != Py_None) {
            refuse(PyExc_ValueError, "q_out without q");
        }
        const int interleaved = PyObject_IsTrue(a[8]);
        if (interleaved < 0) throw Refused{};
        const On on(cache.dev);
        const int rc = litetopk_kv_append(&c, &b, k.data_ptr(), v.data_ptr(), q, T, Hq, f, rot, interleaved, q_out, on.stream);
        if (rc != LTK_OK) failed(rc, "litetopk_kv_append");
        cache.written();
        if (q_o == Py_None) Py_RETURN_NONE;
        if (qo_o == Py_None) return THPVariable_Wrap(qo);
        in_place(qo);
        Py_INCREF(qo_o);
        return qo_o;
    });
}

PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 10);
        Call x(a[1], a[2], a[3], a[4], a[0], a[5], a[8]);
        const int window = int32_of(a[6], "window"), n_sink = int32_of(a[7], "n_sink");
        x.workspace(LTK_ATTEND, (int64_t)x.batch.max_pages * x.cache.c.page_size, 0, a[9]);
        const On on(x.cache.dev);
        return x.result(litetopk_attend(&x.cache.c, &x.batch, x.q, x.T, x.Hq, x.scale, window, n_sink, x.out.data_ptr(),
                                        x.ws_at, x.ws_bytes, on.stream),
                        "litetopk_attend", a[8]);
    });
}

PyObject* attend_selected(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 9);
        Call x(a[1], a[2], a[3], a[4], a[0], a[6], a[7]);
        const at::Tensor& idx = tensor(a[5], "idx", kI32, {x.T, -1}, x.cache.dev);
        const int64_t topk = idx.size(1);
        if (topk < 1 || topk > 65536)
            refuse(PyExc_ValueError, "idx must hold 1 to 65536 keys a row, got " + std::to_string(topk));
        x.workspace(LTK_ATTEND_SELECTED, topk, 0, a[8]);
        const On on(x.cache.dev);
        return x.result(litetopk_attend_selected(&x.cache.c, &x.batch, x.q, x.T, x.Hq,
                                                 static_cast<const int32_t*>(idx.data_ptr()), (int32_t)topk, x.scale,
                                                 x.out.data_ptr(), x.ws_at, x.ws_bytes, on.stream),
                        "litetopk_attend_selected", a[7]);
    });
}

PyObject* attend_packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 11);
        Call x(a[1], a[2], nullptr, a[3], a[0], a[8], a[9]);
        if (x.batch.n_seq != 1)
            refuse(PyExc_ValueError, "attend_packed takes one sequence, got " + std::to_string(x.batch.n_seq));
        const int group = int32_of(a[7], "group");
        if (group < 1 || group > 32) refuse(PyExc_ValueError, "group must lie in 1 .. 32, got " + std::to_string(group));
        const int64_t ng = ((int64_t)x.T + group - 1) / group;
        const at::Tensor& sh = tensor(a[4], "shared", kI32, {ng, -1}, x.cache.dev);
        const int64_t cap = sh.size(1);
        if (cap < 1 || cap > (1 << 26))
            refuse(PyExc_ValueError, "shared must hold 1 to 2^26 entries a group, got " + std::to_string(cap));
        const at::Tensor& mk = tensor(a[5], "masks", kU32, {ng, cap}, x.cache.dev);
        const at::Tensor& ln = tensor(a[6], "lens", kI32, {ng}, x.cache.dev);
        x.workspace(LTK_ATTEND_PACKED, cap, group, a[10]);
        const On on(x.cache.dev);
        return x.result(litetopk_attend_packed(&x.cache.c, &x.batch, x.q, x.T, x.Hq,
                                               static_cast<const int32_t*>(sh.data_ptr()),
                                               static_cast<const uint32_t*>(mk.data_ptr()),
                                               static_cast<const int32_t*>(ln.data_ptr()), group, (int32_t)cap, x.scale,
                                               x.out.data_ptr(), x.ws_at, x.ws_bytes, on.stream),
                        "litetopk_attend_packed", a[9]);
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr
PyMethodDef kMethods[] = {{"kv_append", FAST(kv_append)},
                          {"attend", FAST(attend)},
                          {"attend_selected", FAST(attend_selected)},
                          {"attend_packed", FAST(attend_packed)},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "ltk_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ltk_bind(void) { return PyModule_Create(&kModule); }
