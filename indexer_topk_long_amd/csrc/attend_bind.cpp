// attend_bind.cpp -- Python entry of the paged cache's operators.
//
// A decode step's calls take a few microseconds on the GPU, as long as reading
// ten tensors' attributes from Python takes.  This module does that reading,
// the checks and the launches: every function takes positional arguments in
// the order of its wrapper in attention.py, which documents them.
#include "bind.hpp"

using namespace ltk_bind;

namespace {

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
            own_workspace(need);
        } else {
            if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "workspace must be a tensor");
            ws = THPVariable_Unpack(o);
            ws_bytes = (size_t)ws.numel() * ws.element_size();
            if (!ws.is_cuda() || !ws.is_contiguous() || ws.get_device() != cache.dev)
                refuse(PyExc_ValueError, "workspace must be a contiguous tensor on the cache's device");
        }
        ws_at = ws.data_ptr();
    }

    void own_workspace(size_t need) {
        // (sizes the library does not take: it says so itself, before it looks at the workspace)
        ws_bytes = need ? need : 256;
        ws = at::empty({(int64_t)ws_bytes}, on_device(cache.dev, at::kByte));
        ws_at = ws.data_ptr();
    }

    PyObject* result(int rc, const char* where, PyObject* out_o, const char* sizes = "attend_workspace_bytes") {
        if (rc == LTK_EWORKSPACE)
            refuse(PyExc_ValueError, "workspace too small: " + std::to_string(ws_bytes) +
                                         " bytes (" + sizes + " gives what suffices)");
        if (rc != LTK_OK) failed(rc, where);
        if (own_out) return THPVariable_Wrap(out);
        in_place(out);
        Py_INCREF(out_o);
        return out_o;
    }
};

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

PyObject* attend_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 10);
        Call x(a[1], a[2], a[3], a[4], a[0], a[7], a[8]);
        const at::Tensor& sl = tensor(a[6], "shared_len", kI32, {-1}, x.cache.dev);
        const int32_t ng = size32(sl.size(0), "shared_len");
        const at::Tensor& gr = tensor(a[5], "groups", kI32, {(int64_t)ng + 1}, x.cache.dev);
        const ltk_kv_cache& c = x.cache.c;
        if (a[9] == Py_None) {
            const size_t need = litetopk_attend_shared_workspace_bytes(x.T, x.Hq, c.n_kv_heads, c.head_dim, x.batch.n_seq, ng,
                                                                       (int64_t)x.batch.max_pages * c.page_size);
            x.own_workspace(need);
        } else {
            x.workspace(LTK_ATTEND, 0, 0, a[9]);
        }
        const On on(x.cache.dev);
        return x.result(litetopk_attend_shared(&c, &x.batch, x.q, x.T, x.Hq, static_cast<const int32_t*>(gr.data_ptr()),
                                               static_cast<const int32_t*>(sl.data_ptr()), ng, x.scale, x.out.data_ptr(),
                                               x.ws_at, x.ws_bytes, on.stream),
                        "litetopk_attend_shared", a[8], "attend_shared_workspace_bytes");
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr
PyMethodDef kMethods[] = {{"kv_append", FAST(kv_append)},
                          {"attend", FAST(attend)},
                          {"attend_selected", FAST(attend_selected)},
                          {"attend_packed", FAST(attend_packed)},
                          {"attend_shared", FAST(attend_shared)},
                          {"attend_prompt", FAST(ltk_bind::attend_prompt)},
                          {"kv_read", FAST(ltk_bind::kv_read)},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "ltk_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ltk_bind(void) { return PyModule_Create(&kModule); }
