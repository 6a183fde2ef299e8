// prompt_bind.cpp -- Python entry of the prompts' operators: functions take
// positional arguments in the order of their wrappers in prompt.py, which
// documents them.
#include "bind.hpp"

#include <c10/hip/HIPGraphsC10Utils.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/variable.h>

#include <memory>
#include <unordered_set>
#include <vector>

namespace ltk_bind {

namespace {

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// A device tensor [rows, heads, D] in 16 bits, whatever its strides are.
const at::Tensor& rows_tensor(PyObject* o, const char* name, const at::Tensor* like, int64_t heads, int64_t D) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    const auto type = t.scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf)
        refuse(PyExc_TypeError, std::string(name) + " must be torch.bfloat16 or torch.float16, got " + c10::toString(type));
    if (like && type != like->scalar_type())
        refuse(PyExc_TypeError, std::string(name) + " is " + c10::toString(type) + ", q is " + c10::toString(like->scalar_type()));
    const auto s = t.sizes();
    if (s.size() != 3 || (heads >= 0 && s[1] != heads) || (D >= 0 && s[2] != D))
        refuse(PyExc_ValueError, std::string(name) + " must be [*, " + (heads < 0 ? "*" : std::to_string(heads)) + ", " +
                                     (D < 0 ? "*" : std::to_string(D)) + "], got " + shape_text(s));
    if (!t.is_cuda() || t.layout() != at::kStrided) refuse(PyExc_ValueError, std::string(name) + " must be a device tensor");
    if (like && t.get_device() != like->get_device())
        refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", q on cuda:" +
                                     std::to_string(like->get_device()) + ": all tensors must share one device");
    if (t.unsafeGetTensorImpl()->_fw_grad(0, t).defined())
        refuse(PyExc_RuntimeError, std::string(name) + " carries a tangent: attend_prompt has no forward derivative");
    return t;
}

// Rows as the library takes them; other strides, and values that wait for their
// negation, are laid out anew, in `held`.
ltk_rows rows_of(const at::Tensor& t, at::Tensor& held) {
    constexpr int64_t kRow = 1 << 23, kHead = 1 << 27;
    held = t;
    const int64_t r = t.size(0) > 1 ? t.stride(0) : 0, h = t.size(1) > 1 ? t.stride(1) : 0;
    const bool fits = !t.is_neg() && (t.size(2) <= 1 || t.stride(2) == 1) && r % 8 == 0 && h % 8 == 0 && r <= kRow && h <= kHead &&
                      ((uintptr_t)t.data_ptr() & 15u) == 0;
    if (!fits && t.numel() > 0) {
        held = t.resolve_neg().contiguous();
        // (contiguous already, but not aligned)
        if (((uintptr_t)held.data_ptr() & 15u) != 0) held = held.clone();
        // (not its own strides: those of dimensions of size 1 stay what they were)
        return {held.data_ptr(), t.size(0) > 1 ? t.size(1) * t.size(2) : 0, t.size(2)};
    }
    return {t.data_ptr(), r, h};
}

struct Shape {
    ltk_prompt p;
    int dev;
};
Shape shape_of(const at::Tensor& q, const at::Tensor& k, const at::Tensor& cu, const at::Tensor& cu_k, double scale, int64_t window) {
    Shape s;
    s.dev = q.get_device();
    s.p.cu = static_cast<const int32_t*>(cu.data_ptr());
    s.p.cu_k = cu_k.defined() ? static_cast<const int32_t*>(cu_k.data_ptr()) : nullptr;
    s.p.n_seq = (int32_t)(cu.size(0) - 1);
    s.p.T = (int32_t)q.size(0);
    s.p.S = (int32_t)k.size(0);
    s.p.n_q_heads = (int32_t)q.size(1);
    s.p.n_kv_heads = (int32_t)k.size(1);
    s.p.head_dim = (int32_t)q.size(2);
    s.p.type = q.scalar_type() == at::kBFloat16 ? LTK_ROWS_BF16 : LTK_ROWS_FP16;
    s.p.scale = (float)scale;
    s.p.window = (int32_t)window;
    return s;
}

// What the library returned other than LTK_OK.
struct Status {
    int rc;
    const char* where;
};

void forward_call(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& cu, const at::Tensor& cu_k,
                  double scale, int64_t window, bool with_lse, at::Tensor& out, at::Tensor& lse, at::Tensor* rest = nullptr) {
    const Shape s = shape_of(q, k, cu, cu_k, scale, window);
    const On on(s.dev);
    at::Tensor held[3];
    const ltk_rows qr = rows_of(q, held[0]), kr = rows_of(k, held[1]), vr = rows_of(v, held[2]);
    out = at::empty({s.p.T, s.p.n_q_heads, s.p.head_dim}, q.options().memory_format(c10::nullopt));
    if (rest) *rest = at::empty_like(out);
    if (with_lse) lse = at::empty({s.p.T, s.p.n_q_heads}, q.options().dtype(at::kFloat));
    const size_t need = litetopk_attend_prompt_workspace_bytes(&s.p, 0);
    // (sizes the library does not take: it says so itself, before it looks at the workspace)
    const at::Tensor ws = at::empty({(int64_t)(need ? need : 256)}, on_device(s.dev, at::kByte));
    const int rc = litetopk_attend_prompt(&s.p, &qr, &kr, &vr, out.data_ptr(), rest ? rest->data_ptr() : nullptr, with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                                          ws.data_ptr(), need ? need : 256, on.stream);
    if (rc != LTK_OK) throw Status{rc, "litetopk_attend_prompt"};
}

struct PromptFn : public torch::autograd::Function<PromptFn> {
    static variable_list forward(AutogradContext* ctx, const at::Tensor& q, const at::Tensor& k, const at::Tensor& v,
                                 const at::Tensor& cu, const std::optional<at::Tensor>& cu_k_, double scale, int64_t window) {
        const at::Tensor cu_k = cu_k_.value_or(at::Tensor());
        at::Tensor out, lse, rest;
        forward_call(q, k, v, cu, cu_k, scale, window, true, out, lse, &rest);
        ctx->save_for_backward({q, k, v, cu, cu_k, out, lse, rest});
        ctx->saved_data["scale"] = scale;
        ctx->saved_data["window"] = window;
        ctx->set_materialize_grads(false);
        ctx->mark_non_differentiable({lse});
        return {out, lse};
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads) {
        TORCH_CHECK(!c10::GradMode::is_enabled(), "attend_prompt has no second derivative (create_graph=True)");
        variable_list none(7);
        if (!grads[0].defined()) return none;
        const auto saved = ctx->get_saved_variables();
        const at::Tensor &q = saved[0], &k = saved[1], &v = saved[2], &out = saved[5], &lse = saved[6], &rest = saved[7];
        const Shape s = shape_of(q, k, saved[3], saved[4], ctx->saved_data["scale"].toDouble(), ctx->saved_data["window"].toInt());
        const On on(s.dev);
        at::Tensor held[4], dq, dk, dv;
        const ltk_rows qr = rows_of(q, held[0]), kr = rows_of(k, held[1]), vr = rows_of(v, held[2]), dr = rows_of(grads[0], held[3]);
        const bool keys = ctx->needs_input_grad(1) || ctx->needs_input_grad(2);
        if (ctx->needs_input_grad(0)) dq = at::empty(q.sizes(), q.options());
        if (keys) dk = at::empty(k.sizes(), k.options()), dv = at::empty(v.sizes(), v.options());
        const size_t need = litetopk_attend_prompt_workspace_bytes(&s.p, 1);
        const at::Tensor ws = at::empty({(int64_t)need}, on_device(s.dev, at::kByte));
        auto at_or_null = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
        const int rc = litetopk_attend_prompt_backward(&s.p, &qr, &kr, &vr, out.data_ptr(), rest.data_ptr(), static_cast<const float*>(lse.data_ptr()),
                                                       &dr, at_or_null(dq), at_or_null(dk), at_or_null(dv), ws.data_ptr(), need,
                                                       on.stream);
        TORCH_CHECK(rc == LTK_OK, "litetopk_attend_prompt_backward: status ", rc);
        none[0] = dq;
        if (ctx->needs_input_grad(1)) none[1] = dk;
        if (ctx->needs_input_grad(2)) none[2] = dv;
        return none;
    }
};

// While a stream is captured, the backward pass of a leaf whose accumulator was
// made on the default stream (by an eager graph that still lives) would make that
// stream, which cannot be part of a capture, wait for it, and end the process:
// refused here, before anything is enqueued.  (Accumulators of other streams, as a
// warm-up leaves them, join the capture.)
void leaves_of_capture(const at::Tensor& t, const char* name) {
    if (!t.requires_grad()) return;
    std::vector<std::shared_ptr<torch::autograd::Node>> todo;
    std::unordered_set<torch::autograd::Node*> seen;
    todo.push_back(t.grad_fn() ? t.grad_fn() : torch::autograd::impl::try_get_grad_accumulator(t));
    while (!todo.empty()) {
        const auto node = todo.back();
        todo.pop_back();
        if (!node || !seen.insert(node.get()).second) continue;
        const auto st = node->num_outputs() == 0 ? node->stream() : std::nullopt;   // an accumulator
        if (st && st->id() == 0)
            refuse(PyExc_RuntimeError, std::string(name) + " depends on a leaf of a graph of the default stream that is still alive: a "
                                                           "backward pass captured now would end the process (drop that graph's "
                                                           "results, warm up on another stream, or call under torch.no_grad())");
        for (const auto& e : node->next_edges()) todo.push_back(e.function);
    }
}

const at::Tensor& offsets(PyObject* o, const char* name, int64_t n, int dev) {
    const at::Tensor& t = tensor(o, name, kI32, {n}, dev);
    if (t.size(0) < 1) refuse(PyExc_ValueError, std::string(name) + " must hold one more entry than there are sequences");
    size32(t.size(0), name);
    return t;
}

}  // namespace

PyObject* attend_prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 8);
        const at::Tensor q = rows_tensor(a[0], "q", nullptr, -1, -1);
        const at::Tensor k = rows_tensor(a[1], "k", &q, -1, q.size(2));
        const at::Tensor v = rows_tensor(a[2], "v", &q, k.size(1), q.size(2));
        if (v.size(0) != k.size(0))
            refuse(PyExc_ValueError, "k has " + std::to_string(k.size(0)) + " rows, v " + std::to_string(v.size(0)));
        const int dev = q.get_device();
        size32(q.size(0), "q"), size32(q.size(1), "q"), size32(q.size(2), "q"), size32(k.size(0), "k"), size32(k.size(1), "k");
        if (k.size(1) < 1 || q.size(1) < 1 || q.size(1) % k.size(1) != 0)
            refuse(PyExc_ValueError, "q has " + std::to_string(q.size(1)) + " heads, k " + std::to_string(k.size(1)) +
                                         ": not a multiple");
        const at::Tensor cu = offsets(a[3], "cu", -1, dev);
        at::Tensor cu_k;
        if (a[4] != Py_None) cu_k = offsets(a[4], "cu_k", cu.size(0), dev);
        if (!cu_k.defined() && k.size(0) != q.size(0))
            refuse(PyExc_ValueError, "without cu_k, k must have q's " + std::to_string(q.size(0)) + " rows, got " +
                                         std::to_string(k.size(0)));
        double scale = 1.0 / sqrt((double)(q.size(2) > 0 ? q.size(2) : 1));
        if (a[5] != Py_None) {
            scale = PyFloat_AsDouble(a[5]);
            if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
        }
        const int window = int32_of(a[6], "window");
        const int with_lse = PyObject_IsTrue(a[7]);
        if (with_lse < 0) throw Refused{};
        at::Tensor out, lse;
        try {
            if (c10::GradMode::is_enabled() && (q.requires_grad() || k.requires_grad() || v.requires_grad())) {
                {
                    const On on(dev);
                    if (c10::hip::currentStreamCaptureStatusMayInitCtx() != c10::hip::CaptureStatus::None) {
                        leaves_of_capture(q, "q");
                        leaves_of_capture(k, "k");
                        leaves_of_capture(v, "v");
                    }
                }
                const variable_list r = PromptFn::apply(q, k, v, cu, cu_k.defined() ? std::optional<at::Tensor>(cu_k) : std::nullopt, scale,
                                                       (int64_t)window);
                out = r[0], lse = r[1];
            } else {
                c10::AutoGradMode off(false);
                forward_call(q, k, v, cu, cu_k, scale, window, with_lse, out, lse);
            }
        } catch (const Status& s) {
            failed(s.rc, s.where);
        }
        if (!with_lse) return THPVariable_Wrap(out);
        PyObject* pair[2] = {THPVariable_Wrap(out), THPVariable_Wrap(lse)};
        PyObject* r = pair[0] && pair[1] ? PyTuple_Pack(2, pair[0], pair[1]) : nullptr;
        Py_XDECREF(pair[0]);
        Py_XDECREF(pair[1]);
        return r;
    });
}

PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        expect_args(n, 7);
        const Cache cache = cache_of(a[0]);
        const ltk_kv_cache& c = cache.c;
        const ltk_kv_batch b = batch_of(a[1], a[2], a[3], cache.dev);
        const int T = int32_of(a[4], "T");
        if (T < 0) refuse(PyExc_ValueError, "T must not be negative, got " + std::to_string(T));
        if (!THPDtype_Check(a[5])) refuse(PyExc_TypeError, "dtype must be a torch.dtype");
        const at::ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
        const Kind kind = type == at::kBFloat16 ? kBf16 : type == at::kHalf ? Kind{at::kHalf, "torch.float16"} : kF32;
        if (type != kind.type)
            refuse(PyExc_TypeError, std::string("dtype must be torch.bfloat16, torch.float16 or torch.float32, got ") + c10::toString(type));
        at::Tensor out[2];
        const bool own = a[6] == Py_None;
        if (own) {
            for (at::Tensor& t : out) t = at::empty({T, c.n_kv_heads, c.head_dim}, on_device(cache.dev, type));
        } else {
            if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 2) refuse(PyExc_TypeError, "out must be a pair of tensors (k, v)");
            out[0] = tensor(PyTuple_GET_ITEM(a[6], 0), "out k", kind, {T, c.n_kv_heads, c.head_dim}, cache.dev);
            out[1] = tensor(PyTuple_GET_ITEM(a[6], 1), "out v", kind, {T, c.n_kv_heads, c.head_dim}, cache.dev);
            const auto ka = (uintptr_t)out[0].data_ptr(), va = (uintptr_t)out[1].data_ptr();
            if ((ka < va ? va - ka : ka - va) < out[0].nbytes())
                refuse(PyExc_ValueError, "out k and out v share memory");
        }
        const On on(cache.dev);
        const int rc = litetopk_kv_read(&c, &b, T, type == at::kBFloat16 ? LTK_ROWS_BF16 : type == at::kHalf ? LTK_ROWS_FP16 : LTK_ROWS_FP32,
                                        out[0].data_ptr(), out[1].data_ptr(), on.stream);
        if (rc != LTK_OK) failed(rc, "litetopk_kv_read");
        if (!own) {
            in_place(out[0]);
            in_place(out[1]);
            Py_INCREF(a[6]);
            return a[6];
        }
        PyObject* pair[2] = {THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1])};
        PyObject* r = pair[0] && pair[1] ? PyTuple_Pack(2, pair[0], pair[1]) : nullptr;
        Py_XDECREF(pair[0]);
        Py_XDECREF(pair[1]);
        return r;
    });
}

}  // namespace ltk_bind
