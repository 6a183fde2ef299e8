// bind.hpp -- what the compiled Python entries share: reading and checking
// arguments, errors, the device and its stream.
#pragma once

#ifndef PY_SSIZE_T_CLEAN
#define PY_SSIZE_T_CLEAN
#endif
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <math.h>

#include <string>

#include "litetopk_prompt.h"

namespace ltk_bind {

// Thrown after a Python error has been set.
struct Refused {};

[[noreturn]] inline void refuse(PyObject* type, const std::string& msg) {
    PyErr_SetString(type, msg.c_str());
    throw Refused{};
}

[[noreturn]] inline void failed(int status, const char* where) {
    PyObject* mod = PyImport_ImportModule("indexer_topk_long_amd._binding");
    PyObject* cls = mod ? PyObject_GetAttrString(mod, "LtkError") : nullptr;
    PyObject* err = cls ? PyObject_CallFunction(cls, "is", status, where) : nullptr;
    if (err) PyErr_SetObject(cls, err);
    Py_XDECREF(err);
    Py_XDECREF(cls);
    Py_XDECREF(mod);
    throw Refused{};
}

inline std::string shape_text(c10::IntArrayRef s) {
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
inline void without_grad(const at::Tensor& t, const char* name) {
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse(PyExc_RuntimeError, std::string(name) + " requires grad: the paged cache's operators are forward only "
                                                       "(call them under torch.no_grad(), or detach it)");
    if (t.unsafeGetTensorImpl()->_fw_grad(0, t).defined())   // (read in place: as an operator it goes through the dispatcher)
        refuse(PyExc_RuntimeError, std::string(name) + " carries a tangent: the paged cache's operators are forward only");
}

// After a call has written a tensor in place: autograd sees that what it saved
// of it has changed.  (Inference tensors count no versions.)
inline void in_place(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A contiguous device tensor of this type and shape (-1: any size), on the
// cache's device where dev >= 0.
inline const at::Tensor& tensor(PyObject* o, const char* name, Kind kind, std::initializer_list<int64_t> want, int dev) {
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
    if (t.is_neg()) refuse(PyExc_ValueError, std::string(name) + " is a view of negated values: resolve_neg() lays them out");
    if (dev >= 0 && t.get_device() != dev)
        refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the cache on cuda:" +
                                     std::to_string(dev) + ": all tensors must share one device");
    return t;
}

inline int int32_of(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
    return (int)v;
}

inline int32_t size32(int64_t n, const char* name) {
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
inline Cache cache_of(PyObject* o) {
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
inline ltk_kv_batch batch_of(PyObject* page_table, PyObject* cu, PyObject* kv_len, int dev) {
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

inline at::TensorOptions on_device(int dev, at::ScalarType t) {
    return at::TensorOptions().dtype(t).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
}

inline void expect_args(Py_ssize_t n, Py_ssize_t want) {
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

// Entries of prompt_bind.cpp.
PyObject* attend_prompt(PyObject*, PyObject* const*, Py_ssize_t);
PyObject* kv_read(PyObject*, PyObject* const*, Py_ssize_t);

}  // namespace ltk_bind
