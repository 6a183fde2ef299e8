// attend_api.hip -- the C ABI declared in include/litetopk_attend.h: argument
// checks and launches on the caller's stream.
#include <math.h>

#include "attend.hpp"

using namespace ltk;

namespace {

// Positions of a table: key offsets past a tile's end stay in 32 bits.
constexpr int64_t kMaxTokens = 0x7fffffff - 127;
// Rows times query heads: a unit's rows past the last one stay in 32 bits.
constexpr int64_t kMaxRows = 0x7fffffff - 255;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }

// Sizes and pointers of the cache and the batch; T rows.
int check_cache(const ltk_kv_cache* c, const ltk_kv_batch* b, int32_t T, bool need_cu, KvCache& kc, KvBatch& kb) {
    if (!c || !b || T < 0) return LTK_EINVAL;
    if (c->n_pages < 1 || c->n_kv_heads < 1 || b->n_seq < 0 || b->max_pages < 1) return LTK_EINVAL;
    if (c->head_dim != 64 && c->head_dim != 128) return LTK_EUNSUPPORTED;
    const int sh = page_shift(c->page_size);
    if (sh < 0) return LTK_EUNSUPPORTED;
    constexpr int64_t kMost = 0x7fffffff;
    if ((int64_t)c->n_pages * c->n_kv_heads > (kMost >> sh) || b->max_pages > (kMaxTokens >> sh)) return LTK_EINVAL;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !aligned16(c->k) || !aligned16(c->v)) return LTK_EINVAL;
    if (T > 0 && b->n_seq > 0 && (!b->page_table || !b->kv_len || (need_cu && !b->cu))) return LTK_EINVAL;
    kc = KvCache{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale,
                 c->n_pages, c->n_kv_heads, sh};
    kb = KvBatch{b->page_table, b->cu, b->kv_len, b->n_seq, b->max_pages};
    return LTK_OK;
}

int check_heads(int32_t T, int32_t Hq, int32_t Hkv) {
    if (Hq < 1 || Hq % Hkv != 0) return LTK_EINVAL;
    return (int64_t)T * Hq > kMaxRows ? LTK_EINVAL : LTK_OK;
}

// A group's (row, head) pairs of a key/value head, which the kernels number.
bool group_fits(int32_t group, int32_t Hq, int32_t Hkv) { return (int64_t)group * (Hq / Hkv) <= 1 << 30; }

int run_attend(int kind, const ltk_kv_cache* cache, AttendArgs& a, int64_t entries, void* ws, size_t ws_bytes,
               void* stream) {
    const AttendPlan p = attend_plan(kind, a.T, a.Hq, a.c.Hkv, cache->head_dim, a.bt.n_seq, entries, a.group);
    if (!p.fits()) return LTK_EINVAL;
    if (ws_bytes < p.ws_bytes) return LTK_EWORKSPACE;
    if (a.T == 0 || a.bt.n_seq == 0) return LTK_OK;
    const int st = litetopk_device_check();
    if (st != LTK_OK) return st;
    return launch_attend(kind, cache->head_dim, p, a, ws, static_cast<hipStream_t>(stream)) == hipSuccess ? LTK_OK
                                                                                                          : LTK_EHIP;
}

// The arguments every attend call shares.
int attend_args(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* q, int32_t T, int32_t Hq, float scale,
                void* out, void* ws, bool need_cu, AttendArgs& a) {
    int st = check_cache(cache, batch, T, need_cu, a.c, a.bt);
    if (st != LTK_OK) return st;
    if ((st = check_heads(T, Hq, cache->n_kv_heads)) != LTK_OK) return st;
    if (T > 0 && (!q || !out || !ws)) return LTK_EINVAL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(ws)) return LTK_EINVAL;
    a.q = static_cast<const uint16_t*>(q);
    a.out = static_cast<uint16_t*>(out);
    a.T = T;
    a.Hq = Hq;
    a.G = Hq / cache->n_kv_heads;
    a.c2 = scale * 1.4426950408889634f;
    return isfinite(a.c2) ? LTK_OK : LTK_EINVAL;
}

}  // namespace

extern "C" {

int litetopk_kv_append(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* k, const void* v,
                       const void* q, int32_t T, int32_t Hq, const double* inv_freq, int32_t rot_dim,
                       int32_t interleaved, void* q_out, void* stream) {
    KvCache kc;
    KvBatch kb;
    int st = check_cache(cache, batch, T, true, kc, kb);
    if (st != LTK_OK) return st;
    if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 2 != 0 || (rot_dim > 0 && !inv_freq)) return LTK_EINVAL;
    if ((q == nullptr) != (q_out == nullptr)) return LTK_EINVAL;
    if (q && (st = check_heads(T, Hq, cache->n_kv_heads)) != LTK_OK) return st;
    if (T > 0 && (!k || !v)) return LTK_EINVAL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || ((uintptr_t)inv_freq & 7u))
        return LTK_EINVAL;
    if (T == 0 || kb.n_seq == 0) return LTK_OK;
    if (!q) Hq = 1;
    const AppendPlan p = append_plan(T, Hq, kc.Hkv, cache->head_dim, kb.n_seq, cache->page_size, rot_dim, q != nullptr);
    if (!p.fits) return LTK_EINVAL;
    if ((st = litetopk_device_check()) != LTK_OK) return st;
    if (launch_kv_append(p, kc, kb, cache->head_dim, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                         static_cast<const uint16_t*>(q), T, Hq, inv_freq, rot_dim, interleaved != 0,
                         static_cast<uint16_t*>(q_out), static_cast<hipStream_t>(stream)) != hipSuccess)
        return LTK_EHIP;
    return LTK_OK;
}

size_t litetopk_attend_workspace_bytes(int32_t kind, int32_t T, int32_t Hq, int32_t n_kv_heads, int32_t head_dim,
                                       int32_t n_seq, int64_t entries, int32_t group) {
    if (kind < LTK_ATTEND || kind > LTK_ATTEND_PACKED || T < 0 || n_kv_heads < 1 || Hq < 1 || Hq % n_kv_heads != 0 ||
        n_seq < 0 || entries < 1 || entries > kMaxTokens || (int64_t)T * Hq > kMaxRows ||
        (head_dim != 64 && head_dim != 128) || (kind == LTK_ATTEND_PACKED && (group < 1 || group > 32 || !group_fits(group, Hq, n_kv_heads))))
        return 0;
    const AttendPlan p = attend_plan(kind, T, Hq, n_kv_heads, head_dim, n_seq, entries, group);
    return p.fits() ? attend_workspace_bound(kind, T, Hq, n_kv_heads, head_dim, n_seq, entries, group) : 0;
}

int litetopk_attend(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* q, int32_t T, int32_t Hq,
                    float scale, int32_t window, int32_t n_sink, void* out, void* ws, size_t ws_bytes, void* stream) {
    AttendArgs a{};
    const int st = attend_args(cache, batch, q, T, Hq, scale, out, ws, true, a);
    if (st != LTK_OK) return st;
    if (window < 0 || n_sink < 0) return LTK_EINVAL;
    a.window = window;
    a.n_sink = window > 0 ? n_sink : 0;
    return run_attend(LTK_ATTEND, cache, a, (int64_t)batch->max_pages * cache->page_size, ws, ws_bytes, stream);
}

int litetopk_attend_selected(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* q, int32_t T,
                             int32_t Hq, const int32_t* idx, int32_t topk, float scale, void* out, void* ws,
                             size_t ws_bytes, void* stream) {
    AttendArgs a{};
    const int st = attend_args(cache, batch, q, T, Hq, scale, out, ws, true, a);
    if (st != LTK_OK) return st;
    if (topk < 1 || topk > 65536 || (T > 0 && !idx)) return LTK_EINVAL;
    a.list = idx;
    a.cap = topk;
    return run_attend(LTK_ATTEND_SELECTED, cache, a, topk, ws, ws_bytes, stream);
}

int litetopk_attend_packed(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* q, int32_t T,
                           int32_t Hq, const int32_t* shared, const uint32_t* masks, const int32_t* lens,
                           int32_t group, int32_t cap, float scale, void* out, void* ws, size_t ws_bytes,
                           void* stream) {
    AttendArgs a{};
    const int st = attend_args(cache, batch, q, T, Hq, scale, out, ws, false, a);
    if (st != LTK_OK) return st;
    if (batch->n_seq != 1 || group < 1 || group > 32 || cap < 1 || cap > (1 << 26)) return LTK_EINVAL;
    if (!group_fits(group, Hq, cache->n_kv_heads)) return LTK_EINVAL;
    if (T > 0 && (!shared || !masks || !lens)) return LTK_EINVAL;
    a.list = shared;
    a.masks = masks;
    a.lens = lens;
    a.group = group;
    a.cap = cap;
    return run_attend(LTK_ATTEND_PACKED, cache, a, cap, ws, ws_bytes, stream);
}

}  // extern "C"
