// prompt_api.hip -- the C ABI declared in include/litetopk_prompt.h: argument
// checks and launches on the caller's stream.
#include <math.h>

#include "prompt.hpp"

using namespace ltk;

namespace {

constexpr int64_t kMaxRows = 0x7fffffff - 255;
// A tile's 64 rows, and the eight heads of a copy, lie within 32 bits of bytes.
constexpr int64_t kMaxRowStride = 1 << 23, kMaxHeadStride = 1 << 27;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int check(const ltk_prompt* p) {
    if (!p || p->n_seq < 0 || p->T < 0 || p->S < 0 || p->n_kv_heads < 1 || p->n_q_heads < 1 ||
        p->n_q_heads % p->n_kv_heads != 0)
        return LTK_EINVAL;
    if ((int64_t)p->T * p->n_q_heads > kMaxRows || (int64_t)p->S * p->n_kv_heads > kMaxRows) return LTK_EINVAL;
    if (p->n_seq > kMaxRows || p->window < 0 || !isfinite(p->scale * 1.4426950408889634f)) return LTK_EINVAL;
    if (p->n_q_heads / p->n_kv_heads >= 1 << 15) return LTK_EINVAL;   // (a group's quotients)
    if (p->head_dim != 64 && p->head_dim != 128) return LTK_EUNSUPPORTED;
    if (p->type != LTK_ROWS_BF16 && p->type != LTK_ROWS_FP16) return LTK_EUNSUPPORTED;
    if (!p->cu_k && p->S != p->T) return LTK_EINVAL;
    return LTK_OK;
}

int rows(const ltk_rows* x, bool used, PrRows& r) {
    if (!x) return LTK_EINVAL;
    if (used && !x->data) return LTK_EINVAL;
    if (!aligned16(x->data) || x->row_stride % 8 || x->head_stride % 8) return LTK_EINVAL;
    if (x->row_stride < 0 || x->row_stride > kMaxRowStride || x->head_stride < 0 || x->head_stride > kMaxHeadStride)
        return LTK_EINVAL;
    r = PrRows{static_cast<const uint16_t*>(x->data), x->row_stride, x->head_stride};
    return LTK_OK;
}

int args(const ltk_prompt* p, const ltk_rows* q, const ltk_rows* k, const ltk_rows* v, PromptArgs& a, PromptPlan& plan) {
    int st = check(p);
    if (st != LTK_OK) return st;
    if ((p->T > 0 || p->S > 0) && !p->cu) return LTK_EINVAL;
    if ((st = rows(q, p->T > 0, a.q)) != LTK_OK || (st = rows(k, p->S > 0, a.k)) != LTK_OK ||
        (st = rows(v, p->S > 0, a.v)) != LTK_OK)
        return st;
    a.cu = p->cu;
    a.cu_k = p->cu_k ? p->cu_k : p->cu;
    a.n_seq = p->n_seq;
    a.T = p->T;
    a.S = p->S;
    a.Hq = p->n_q_heads;
    a.Hkv = p->n_kv_heads;
    a.G = a.Hq / a.Hkv;
    a.div_g = a.G == 1 ? 0u : (uint32_t)(((1ull << 32) + a.G - 1) / a.G);
    a.one_g = a.G == 1 ? ~0u : 0u;
    a.scale = p->scale;
    a.c2 = p->scale * 1.4426950408889634f;
    a.window = p->window;
    plan = prompt_plan(a.T, a.S, a.Hq, a.Hkv, p->head_dim, a.n_seq, a.window);
    return plan.fits ? LTK_OK : LTK_EINVAL;
}

}  // namespace

extern "C" {

size_t litetopk_attend_prompt_workspace_bytes(const ltk_prompt* p, int32_t backward) {
    if (check(p) != LTK_OK) return 0;
    const PromptPlan plan = prompt_plan(p->T, p->S, p->n_q_heads, p->n_kv_heads, p->head_dim, p->n_seq, p->window);
    return !plan.fits ? 0 : backward ? plan.bwd_bytes : plan.fwd_bytes;
}

int litetopk_attend_prompt(const ltk_prompt* p, const ltk_rows* q, const ltk_rows* k, const ltk_rows* v, void* out,
                           void* rest, float* lse, void* ws, size_t ws_bytes, void* stream) {
    PromptArgs a{};
    PromptPlan plan;
    int st = args(p, q, k, v, a, plan);
    if (st != LTK_OK) return st;
    if ((p->T > 0 && (!out || !ws)) || !aligned16(out) || !aligned16(rest) || !aligned16(ws) || ((uintptr_t)lse & 3u)) return LTK_EINVAL;
    if (ws_bytes < plan.fwd_bytes) return LTK_EWORKSPACE;
    if (p->T == 0) return LTK_OK;
    if ((st = litetopk_device_check()) != LTK_OK) return st;
    a.out = static_cast<uint16_t*>(out);
    a.rest = static_cast<uint16_t*>(rest);
    a.lse = lse;
    return launch_prompt(plan, p->type, p->head_dim, a, ws, static_cast<hipStream_t>(stream)) == hipSuccess ? LTK_OK : LTK_EHIP;
}

int litetopk_attend_prompt_backward(const ltk_prompt* p, const ltk_rows* q, const ltk_rows* k, const ltk_rows* v,
                                    const void* out, const void* rest, const float* lse, const ltk_rows* dout,
                                    void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
    PromptArgs a{};
    PromptPlan plan;
    int st = args(p, q, k, v, a, plan);
    if (st != LTK_OK) return st;
    if ((st = rows(dout, p->T > 0, a.dout)) != LTK_OK) return st;
    if (p->T > 0 && (!out || !lse)) return LTK_EINVAL;
    if ((dk == nullptr) != (dv == nullptr)) return LTK_EINVAL;
    if (!aligned16(out) || !aligned16(rest) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(ws) || ((uintptr_t)lse & 3u))
        return LTK_EINVAL;
    if ((p->T > 0 || p->S > 0) && !ws) return LTK_EINVAL;
    if (ws_bytes < plan.bwd_bytes) return LTK_EWORKSPACE;
    if ((p->T == 0 || !dq) && (p->S == 0 || !dk)) return LTK_OK;
    if ((st = litetopk_device_check()) != LTK_OK) return st;
    a.out_in = static_cast<const uint16_t*>(out);
    a.rest_in = static_cast<const uint16_t*>(rest);
    a.lse = const_cast<float*>(lse);
    a.dq = static_cast<uint16_t*>(dq);
    a.dk = static_cast<uint16_t*>(dk);
    a.dv = static_cast<uint16_t*>(dv);
    return launch_prompt_backward(plan, p->type, p->head_dim, a, ws, static_cast<hipStream_t>(stream)) == hipSuccess ? LTK_OK
                                                                                                                   : LTK_EHIP;
}

}  // extern "C"
