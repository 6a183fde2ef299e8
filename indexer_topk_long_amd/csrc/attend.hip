// attend.hip -- attention over the paged e4m3 cache for few rows per key on
// gfx950 (decode, speculative decode, selected keys): bound by reading the
// cache once.
//
// For a query row q and the keys s it sees, with page scales ks and vs,
//   y_s = scale log2(e) ks (q . k_s) + log2(vs)
//   out = sum_s 2^(y_s - m) vbyte_s / sum_s 2^(y_s - m) / vs,
// one pass with a running reference m: moving the value scale into the
// exponent keeps the weights 2^(y - m) within fp16 whatever the scales are,
// and the divisor takes it out again.
//
// A wave takes 32 keys at a time and reads them straight into matrix-core
// operands; no key or value passes through LDS:
//  - scores, transposed (keys on the rows of v_mfma_f32_16x16x32_bf16, query
//    rows on its columns): lane (c, g) = (lane % 16, lane / 16) loads 16-byte
//    pieces of key row c; e4m3 to bf16 is exact;
//  - a score register of lane (c, g) then holds query row c against keys
//    4 g + i, which is the layout the second product wants for its weights:
//    weights are rounded to fp16 in place (e4m3 to fp16 is exact too, and
//    fp16 keeps 3 bits more of a weight than bf16);
//  - values: lane (c, g) loads D / 16 bytes of the 8 keys its weights belong
//    to; pairing keys byte by byte gives, for each e < D / 16, the operand
//    whose row c is dimension c D / 16 + e.
// Softmax statistics stay in the lane: m moves only when a score passes it by
// 2^8, so most tiles need no exchange between lanes; the weights' sums of the
// four lane groups are joined once at the end.
#include <algorithm>

#include "attend.hpp"

namespace ltk {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;            // keys per wave step
constexpr float kNoRef = -1e30f;     // reference before the first visible key
constexpr float kSlack = 8.0f;       // scores may pass the reference by 2^8: weights up to 256 in fp16
constexpr int kListChunk = 2048;     // list entries staged in LDS at a time

__device__ __forceinline__ float max_groups(float x) {   // over the four 16-lane groups
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_groups(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// 8 e4m3 bytes as bf16, exact
__device__ __forceinline__ at_bf16x8 bf16_of(uint32_t a, uint32_t b) {
    const at_bf16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const at_bf16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const at_bf16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const at_bf16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return at_bf16x8{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
}

// The wave's share of 32 keys: halves A (keys 0..15) and B (16..31).
template <int D>
struct KvTile {
    at_u32x4 k[2][D / 64];          // key row c of each half, bytes 64 h + 16 g
    uint32_t v[8][D / 64];          // the lane's 8 keys, bytes c D/16 ..
};

// Per-key constants of one half, for the lane's keys 4 g + i.
struct HalfScale {
    float c[4], lv[4], iv[4];   // scale log2(e) ks, log2(vs), 1 / vs
};

// Running state of 16 query rows: reference, weight sum (of the lane's keys)
// and the D / 16 x 4 accumulators of row c, dimensions (4 g + r) D/16 + e.
template <int D>
struct RowState {
    float m, l;
    at_f32x4 o[D / 16];
};

template <int D>
__device__ __forceinline__ void rescale(RowState<D>& st, float m_new) {
    const float f = __builtin_amdgcn_exp2f(st.m - m_new);
    st.l *= f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) st.o[e] *= f;
    st.m = m_new;
}

// Values as matrix operands: operand e holds byte e of the lane's 8 keys.
template <int D>
__device__ __forceinline__ void value_operands(const KvTile<D>& t, at_f16x8 (&a)[D / 16]) {
#pragma unroll
    for (int w = 0; w < D / 64; ++w)
#pragma unroll
        for (int p = 0; p < 4; ++p) {   // key pair (2p, 2p + 1)
            const uint32_t lo = __builtin_amdgcn_perm(t.v[2 * p + 1][w], t.v[2 * p][w], 0x05010400u);
            const uint32_t hi = __builtin_amdgcn_perm(t.v[2 * p + 1][w], t.v[2 * p][w], 0x07030602u);
            const at_f16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
            const at_f16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
            const at_f16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
            const at_f16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
            a[4 * w + 0][2 * p] = x0[0], a[4 * w + 0][2 * p + 1] = x0[1];
            a[4 * w + 1][2 * p] = x1[0], a[4 * w + 1][2 * p + 1] = x1[1];
            a[4 * w + 2][2 * p] = x2[0], a[4 * w + 2][2 * p + 1] = x2[1];
            a[4 * w + 3][2 * p] = x3[0], a[4 * w + 3][2 * p + 1] = x3[1];
        }
}

// One 32-key tile against MT x 16 query rows.  mask(mt, key) says whether the
// lane's query row of tile mt sees key (0..31) of the tile; called only where
// MASK.
template <int D, int MT, bool MASK, class Mask>
__device__ __forceinline__ void tile_step(const KvTile<D>& t, const at_bf16x8 (&q)[MT][D / 32], const HalfScale (&hs)[2],
                                          RowState<D> (&st)[MT], int g, Mask mask) {
    at_bf16x8 kf[2][D / 32];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            kf[a][2 * h] = bf16_of(t.k[a][h][0], t.k[a][h][1]);
            kf[a][2 * h + 1] = bf16_of(t.k[a][h][2], t.k[a][h][3]);
        }
    at_f16x8 vf[D / 16];
    value_operands<D>(t, vf);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        at_f32x4 s[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            s[a] = at_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                s[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[a][c], q[mt][c], s[a], 0, 0, 0);
        }
        float y[8], top = kNoRef;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = __builtin_fmaf(s[a][i], hs[a].c[i], hs[a].lv[i]);
                if constexpr (MASK) x = mask(mt, 16 * a + 4 * g + i) ? x : -INFINITY;
                y[4 * a + i] = x;
                top = fmaxf(top, x);
            }
        if (__any(top > st[mt].m + kSlack)) rescale<D>(st[mt], fmaxf(st[mt].m, max_groups(top)));
        at_f16x8 p;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float p0 = __builtin_amdgcn_exp2f(y[4 * a + i] - st[mt].m);
                const float p1 = __builtin_amdgcn_exp2f(y[4 * a + i + 1] - st[mt].m);
                st[mt].l = __builtin_fmaf(p0, hs[a].iv[i], st[mt].l);
                st[mt].l = __builtin_fmaf(p1, hs[a].iv[i + 1], st[mt].l);
                const at_f32x2 pp{p0, p1};
                const at_f16x2 ph = __builtin_convertvector(pp, at_f16x2);
                p[4 * a + i] = ph[0], p[4 * a + i + 1] = ph[1];
            }
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
            st[mt].o[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[e], p, st[mt].o[e], 0, 0, 0);
    }
}

// The waves' states joined through LDS, then the unit's rows written: bf16
// rows when the unit has one split, else fp32 partial rows and (m, l).
//   part layout per (unit, split): [16 MT] rows of D floats, then [16 MT] (m, l)
template <int D, int MT, class Row>
__device__ __forceinline__ void finish(const AttendArgs& a, RowState<D> (&st)[MT], float* sh, int64_t slot, int splits,
                                       Row row_of) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    constexpr int kStride = D + 4;   // floats per row in LDS: rows start 4 banks apart
    float* so = sh;                          // [kWaves][16][kStride]
    float* sm = sh + kWaves * 16 * kStride;  // [kWaves][16][2]
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const float l = sum_groups(st[mt].l);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < D / 16; e += 4)
                *reinterpret_cast<at_f32x4*>(so + (wave * 16 + c) * kStride + (4 * g + r) * (D / 16) + e) =
                    at_f32x4{st[mt].o[e][r], st[mt].o[e + 1][r], st[mt].o[e + 2][r], st[mt].o[e + 3][r]};
        if (g == 0) {
            sm[(wave * 16 + c) * 2] = st[mt].m;
            sm[(wave * 16 + c) * 2 + 1] = l;
        }
        __syncthreads();
        // 16 threads per row, D / 16 dimensions each
        const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * (D / 16);
        float m = kNoRef;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sm[(w * 16 + r) * 2]);
        float sum = 0.0f, o[D / 16];
#pragma unroll
        for (int e = 0; e < D / 16; ++e) o[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(sm[(w * 16 + r) * 2] - m);
            sum = __builtin_fmaf(f, sm[(w * 16 + r) * 2 + 1], sum);
            const float* src = so + (w * 16 + r) * kStride + d0;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) o[e] = __builtin_fmaf(f, src[e], o[e]);
        }
        const int64_t row = row_of(mt * 16 + r);   // row * Hq + head, -1 past the unit
        if (row < 0) continue;
        if (splits == 1) {
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            uint32_t w[D / 32];
#pragma unroll
            for (int e = 0; e < D / 16; e += 2) w[e / 2] = pack_bf16(o[e] * inv, o[e + 1] * inv);
            uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + d0);
            if constexpr (D == 128)
                *reinterpret_cast<at_u32x4*>(dst) = at_u32x4{w[0], w[1], w[2], w[3]};
            else
                *reinterpret_cast<at_u32x2*>(dst) = at_u32x2{w[0], w[1]};
        } else {
            float* dst = a.part + slot * (16 * MT) * (D + 2);
#pragma unroll
            for (int e = 0; e < D / 16; e += 4)
                *reinterpret_cast<at_f32x4*>(dst + (size_t)(mt * 16 + r) * D + d0 + e) = at_f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]};
            if ((threadIdx.x & 15) == 0) {
                float* ml = dst + (size_t)16 * MT * D + (mt * 16 + r) * 2;
                ml[0] = m;
                ml[1] = sum;
            }
        }
    }
}

template <int D, int MT>
constexpr size_t finish_lds() {
    return (size_t)(kWaves * 16 * (D + 4) + kWaves * 16 * 2) * 4;
}

// Rows of a dense unit: sequence b's rows times the G query heads of one
// key/value head, flattened as (row, head), 16 MT of them from r0 on.
struct DenseUnit {
    SeqRows sr;
    int b, f0, f1;              // flattened range [f0, f1); empty when f0 >= f1
    int pos_lo, pos_hi;         // positions of its first and last row
    int sink_tiles, win_tile0;  // key tiles: [0, sink_tiles) and from win_tile0 on
    int lo, hi;                 // visible keys: < n_sink (sinks) or in [lo, hi)
    int tiles, per;             // key tiles in all, and per split
};

template <int MT>
__device__ __forceinline__ DenseUnit dense_unit(const AttendArgs& a, int u) {
    constexpr int RT = 16 * MT;
    DenseUnit d;
    d.b = unit_seq(a.bt, u, a.T, a.G, RT, 1);
    d.sr = seq_rows(a.bt, d.b, a.T);
    const int nth = u - unit_first(a.bt, d.b, a.T, a.G, RT, 1);
    const int n = (d.sr.r1 - d.sr.r0) * a.G;
    d.f0 = nth * RT;
    d.f1 = min(d.f0 + RT, n);
    if (nth < 0 || d.f0 >= n) {
        d.f0 = d.f1 = 0;
        return d;
    }
    d.pos_lo = d.sr.pos0 + d.f0 / a.G;
    d.pos_hi = d.sr.pos0 + (d.f1 - 1) / a.G;
    const int cap = a.bt.max_pages << a.c.page_shift;
    d.hi = min(max(d.pos_hi + 1, 0), cap);
    d.lo = a.window > 0 ? min(max(d.pos_lo - a.window + 1, 0), d.hi) : 0;
    const int sinks = a.window > 0 ? min(a.n_sink, d.lo) : 0;
    d.sink_tiles = (sinks + kTile - 1) / kTile;
    d.win_tile0 = max(d.lo / kTile, d.sink_tiles);
    d.tiles = d.sink_tiles + max((d.hi + kTile - 1) / kTile - d.win_tile0, 0);
    // whole rounds of the waves
    d.per = ((d.tiles + a.splits - 1) / a.splits + kWaves - 1) / kWaves * kWaves;
    return d;
}

template <int D, int MT>
__device__ __forceinline__ void load_queries(const AttendArgs& a, at_bf16x8 (&q)[MT][D / 32], int64_t (&row)[MT], int c,
                                             int g) {
    // row[mt]: row * Hq + head of the lane's query row, or -1
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            at_u32x4 w{0u, 0u, 0u, 0u};
            // dimensions 64 (j / 2) + 16 g + 8 (j % 2): the same order as the key pieces
            if (row[mt] >= 0)
                w = *reinterpret_cast<const at_u32x4*>(a.q + row[mt] * D + 64 * (j / 2) + 16 * g + 8 * (j % 2));
            q[mt][j] = __builtin_bit_cast(at_bf16x8, w);
        }
    (void)c;
}

// ------------------------------------------------------------ dense keys

template <int D, int MT>
__global__ __launch_bounds__(64 * kWaves) void attend_kernel(AttendArgs a) {
    extern __shared__ float sh[];
    const int h = blockIdx.x % a.c.Hkv, rest = blockIdx.x / a.c.Hkv;
    const int split = rest % a.splits, u = rest / a.splits;
    const DenseUnit d = dense_unit<MT>(a, u);
    if (d.f0 >= d.f1) return;
    const int t0 = split * d.per, t1 = min(t0 + d.per, d.tiles);
    if (split > 0 && t0 >= t1) return;   // split 0 of a unit that sees nothing writes its zeros
    const int used = max((d.tiles + d.per - 1) / max(d.per, 1), 1);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;

    auto row_of = [&](int r) -> int64_t {
        const int f = d.f0 + r;
        if (f >= d.f1) return -1;
        const int i = f / a.G;
        return (int64_t)(d.sr.r0 + i) * a.Hq + h * a.G + (f - i * a.G);
    };
    at_bf16x8 q[MT][D / 32];
    int64_t row[MT];
    int pos[MT];
    RowState<D> st[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        row[mt] = row_of(mt * 16 + c);
        pos[mt] = row[mt] < 0 ? -1 : d.sr.pos0 + (d.f0 + mt * 16 + c) / a.G;
        st[mt].m = kNoRef;
        st[mt].l = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) st[mt].o[e] = at_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    load_queries<D, MT>(a, q, row, c, g);

    const int32_t* table = a.bt.table + (size_t)d.b * a.bt.max_pages;
    const int page = 1 << a.c.page_shift;
    struct Where {
        int key0, pid[2];   // page of each half, -1 when it has none
    };
    auto where = [&](int t) {
        Where w;
        w.key0 = (t < d.sink_tiles ? t : d.win_tile0 + t - d.sink_tiles) * kTile;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int key = w.key0 + 16 * x, pg = key >> a.c.page_shift;
            const int id = table[min(pg, a.bt.max_pages - 1)];
            // (a page with no visible key is not looked at: its scale and bytes may be anything)
            const bool seen = key < d.hi && (key + 15 >= d.lo || key < a.n_sink);
            w.pid[x] = (seen && id >= 0 && id < a.c.n_pages) ? id : -1;
        }
        return w;
    };
    auto load = [&](KvTile<D>& t, const Where& w) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const size_t base = ((((size_t)max(w.pid[x], 0) * a.c.Hkv + h) << a.c.page_shift) +
                                 ((w.key0 + 16 * x) & (page - 1))) * D;
            const uint8_t* kp = a.c.k + base;
            const uint8_t* vp = a.c.v + base;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                t.k[x][j] = *reinterpret_cast<const at_u32x4*>(kp + c * D + 64 * j + 16 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* p = vp + (4 * g + i) * D + c * (D / 16);
                if constexpr (D == 128) {
                    const at_u32x2 z = *reinterpret_cast<const at_u32x2*>(p);
                    t.v[4 * x + i][0] = z[0];
                    t.v[4 * x + i][1] = z[1];
                } else {
                    t.v[4 * x + i][0] = *reinterpret_cast<const uint32_t*>(p);
                }
            }
        }
    };
    auto step = [&](KvTile<D>& t, const Where& w) {
        HalfScale hs[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const size_t at = (size_t)max(w.pid[x], 0) * a.c.Hkv + h;
            const float ks = w.pid[x] >= 0 ? a.c.ks[at] : 1.0f, vs = w.pid[x] >= 0 ? a.c.vs[at] : 1.0f;
            const float cc = a.c2 * ks, lv = __builtin_amdgcn_logf(vs), iv = 1.0f / vs;   // v_log_f32: base 2
#pragma unroll
            for (int i = 0; i < 4; ++i) hs[x].c[i] = cc, hs[x].lv[i] = lv, hs[x].iv[i] = iv;
        }
        const int last = w.key0 + kTile - 1;
        const bool whole = w.pid[0] >= 0 && w.pid[1] >= 0 && last <= d.pos_lo && last < d.hi &&
                           (a.window <= 0 || w.key0 > d.pos_hi - a.window || last < a.n_sink) && d.f1 - d.f0 == 16 * MT;
        if (whole) {
            tile_step<D, MT, false>(t, q, hs, st, g, [](int, int) { return true; });
            return;
        }
        // bytes of keys that no row sees may be NaN: their weights are 0, so the values must be finite
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = w.key0 + 16 * x + 4 * g + i;
                const bool ok = w.pid[x] >= 0 && key < d.hi && (key >= d.lo || key < a.n_sink);
#pragma unroll
                for (int j = 0; j < D / 64; ++j) t.v[4 * x + i][j] = ok ? t.v[4 * x + i][j] : 0u;
            }
        tile_step<D, MT, true>(t, q, hs, st, g, [&](int mt, int k) {
            const int key = w.key0 + k;
            return (k < 16 ? w.pid[0] : w.pid[1]) >= 0 && key <= pos[mt] && key < d.hi &&
                   (a.window <= 0 || key > pos[mt] - a.window || key < a.n_sink);
        });
    };

    KvTile<D> ta, tb;
    int t = t0 + wave;
    if (t < t1) {
        Where wa = where(t), wb = wa;
        load(ta, wa);
        while (true) {
            const bool more = t + kWaves < t1;
            if (more) wb = where(t + kWaves), load(tb, wb);
            step(ta, wa);
            if (!more) break;
            t += kWaves;
            const bool more2 = t + kWaves < t1;
            if (more2) wa = where(t + kWaves), load(ta, wa);
            step(tb, wb);
            if (!more2) break;
            t += kWaves;
        }
    }
    finish<D, MT>(a, st, sh, ((int64_t)u * a.c.Hkv + h) * a.splits + split, used, row_of);
}

// --------------------------------------------------- listed keys (one row)

// One entry of the staged list: row of the cache for the unit's head, and the
// constants of its page.
struct ListLds {
    int32_t row[kListChunk];
    float c[kListChunk], lv[kListChunk], iv[kListChunk];
};

// A unit is one row of the call (all heads of one key/value head, in tiles of
// 16 MT heads); its list is idx[row], or with PACKED the entries of the row's
// group whose mask holds the row's bit.
template <int D, int MT, bool PACKED>
__global__ __launch_bounds__(64 * kWaves) void attend_list_kernel(AttendArgs a) {
    extern __shared__ float sh[];
    ListLds& ls = *reinterpret_cast<ListLds*>(sh);
    __shared__ int s_cnt[kWaves];
    constexpr int RT = 16 * MT;
    const int h = blockIdx.x % a.c.Hkv;
    int rest = blockIdx.x / a.c.Hkv;
    const int split = rest % a.splits;
    rest /= a.splits;
    const int ht = (a.G + RT - 1) / RT, tile = rest % ht, t = rest / ht;
    int b = 0, pos;
    if constexpr (PACKED) {
        pos = max(a.bt.len[0], 0) - a.T + t;
    } else {
        int hi = a.bt.n_seq - 1;
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if (cu_at(a.bt, mid, a.T) <= t)
                b = mid;
            else
                hi = mid - 1;
        }
        const SeqRows sr = seq_rows(a.bt, b, a.T);
        if (t < sr.r0 || t >= sr.r1) return;
        pos = sr.pos0 + (t - sr.r0);
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int grp = PACKED ? t / a.group : 0, bit = PACKED ? t % a.group : 0;
    const int32_t* list = a.list + (size_t)(PACKED ? grp : t) * a.cap;
    const uint32_t* masks = PACKED ? a.masks + (size_t)grp * a.cap : nullptr;
    const int n = PACKED ? min(max(a.lens[grp], 0), a.cap) : a.cap;
    const int per = (n + a.splits - 1) / a.splits;
    const int e0 = split * per, e1 = min(e0 + per, n);
    if (split > 0 && e0 >= e1) return;
    const int used = max((n + per - 1) / max(per, 1), 1);

    auto row_of = [&](int r) -> int64_t {
        const int head = tile * RT + r;
        return head < a.G ? (int64_t)t * a.Hq + h * a.G + head : -1;
    };
    at_bf16x8 q[MT][D / 32];
    int64_t row[MT];
    RowState<D> st[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        row[mt] = row_of(mt * 16 + c);
        st[mt].m = kNoRef;
        st[mt].l = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) st[mt].o[e] = at_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    load_queries<D, MT>(a, q, row, c, g);
    const int32_t* table = a.bt.table + (size_t)b * a.bt.max_pages;
    const int page = 1 << a.c.page_shift;
    const int end = min(max(pos + 1, 0), a.bt.max_pages << a.c.page_shift);   // keys the row may see

    auto load = [&](KvTile<D>& x, int at) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const uint8_t* kp = a.c.k + (size_t)ls.row[at + 16 * z + c] * D;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) x.k[z][j] = *reinterpret_cast<const at_u32x4*>(kp + 64 * j + 16 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* p = a.c.v + (size_t)ls.row[at + 16 * z + 4 * g + i] * D + c * (D / 16);
                if constexpr (D == 128) {
                    const at_u32x2 y = *reinterpret_cast<const at_u32x2*>(p);
                    x.v[4 * z + i][0] = y[0];
                    x.v[4 * z + i][1] = y[1];
                } else {
                    x.v[4 * z + i][0] = *reinterpret_cast<const uint32_t*>(p);
                }
            }
        }
    };
    auto step = [&](KvTile<D>& x, int at, int cnt) {
        HalfScale hs[2];
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = at + 16 * z + 4 * g + i;
                hs[z].c[i] = ls.c[k], hs[z].lv[i] = ls.lv[k], hs[z].iv[i] = ls.iv[k];
            }
        if (at + kTile <= cnt)
            tile_step<D, MT, false>(x, q, hs, st, g, [](int, int) { return true; });
        else   // padded entries repeat the last key
            tile_step<D, MT, true>(x, q, hs, st, g, [&](int, int k) { return at + k < cnt; });
    };

    for (int c0 = e0; c0 < e1; c0 += kListChunk) {
        // the chunk's keys, compacted in list order
        const int c1 = min(c0 + kListChunk, e1);
        int cnt = 0;
        __syncthreads();   // the previous chunk has been read
        for (int s0 = c0; s0 < c1; s0 += 64 * kWaves) {
            const int e = s0 + threadIdx.x;
            int s = -1;
            if (e < c1) {
                s = list[e];
                if (PACKED && !((masks[e] >> bit) & 1u)) s = -1;
            }
            int pid = -1;
            if (s >= 0 && s < end) {
                pid = table[s >> a.c.page_shift];
                if (pid >= a.c.n_pages) pid = -1;
            }
            const uint64_t have = __ballot(pid >= 0);
            if (lane == 0) s_cnt[wave] = __popcll(have);
            __syncthreads();
            int base = cnt;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                if (w < wave) base += s_cnt[w];
                cnt += s_cnt[w];
            }
            if (pid >= 0) {
                const int at = base + __popcll(have & ((1ull << lane) - 1ull));
                const size_t pg = (size_t)pid * a.c.Hkv + h;
                const float vs = a.c.vs[pg];
                ls.row[at] = (int)((pg << a.c.page_shift) + (s & (page - 1)));
                ls.c[at] = a.c2 * a.c.ks[pg];
                ls.lv[at] = __builtin_amdgcn_logf(vs);
                ls.iv[at] = 1.0f / vs;
            }
            __syncthreads();
        }
        if (cnt == 0) continue;
        // pad the last tile with its last key (read, never counted)
        const int padded = (cnt + kTile - 1) / kTile * kTile;
        if ((int)threadIdx.x < padded - cnt) {
            const int at = cnt + threadIdx.x;
            ls.row[at] = ls.row[cnt - 1];
            ls.c[at] = ls.c[cnt - 1], ls.lv[at] = ls.lv[cnt - 1], ls.iv[at] = ls.iv[cnt - 1];
        }
        __syncthreads();
        KvTile<D> ta, tb;
        int at = wave * kTile;
        constexpr int kStep = kWaves * kTile;
        if (at < cnt) {
            load(ta, at);
            while (true) {
                const bool more = at + kStep < cnt;
                if (more) load(tb, at + kStep);
                step(ta, at, cnt);
                if (!more) break;
                at += kStep;
                const bool more2 = at + kStep < cnt;
                if (more2) load(ta, at + kStep);
                step(tb, at, cnt);
                if (!more2) break;
                at += kStep;
            }
        }
    }
    __syncthreads();   // the list is done with: finish() reuses its LDS
    const int64_t unit = ((int64_t)t * ht + tile) * a.c.Hkv + h;
    finish<D, MT>(a, st, sh, unit * a.splits + split, used, row_of);
}

// ------------------------------------------------------- joining the splits

// One workgroup per query row and head: 256 threads = 256 / (D / 4) groups
// that take splits in turn, then one sum over the groups.
template <int D, int MT, int KIND>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
    constexpr int RT = 16 * MT, kLanes = D / 4, kGroups = 256 / kLanes;
    __shared__ float s_o[kGroups][D + 4];
    __shared__ float s_ml[kGroups][2];
    const int64_t r = blockIdx.x;   // row * Hq + head
    const int t = (int)(r / a.Hq), head = (int)(r % a.Hq), h = head / a.G, g = head - h * a.G;
    int64_t unit;
    int used, at;
    if constexpr (KIND == LTK_ATTEND) {
        int b = 0, hi = a.bt.n_seq - 1;
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if (cu_at(a.bt, mid, a.T) <= t)
                b = mid;
            else
                hi = mid - 1;
        }
        const SeqRows sr = seq_rows(a.bt, b, a.T);
        if (t < sr.r0 || t >= sr.r1) return;
        const int f = (t - sr.r0) * a.G + g, u = unit_first(a.bt, b, a.T, a.G, RT, 1) + f / RT;
        const DenseUnit d = dense_unit<MT>(a, u);
        unit = (int64_t)u * a.c.Hkv + h;
        used = (d.tiles + d.per - 1) / max(d.per, 1);
        at = f % RT;
    } else {
        if constexpr (KIND == LTK_ATTEND_SELECTED) {
            if (t < cu_at(a.bt, 0, a.T) || t >= cu_at(a.bt, a.bt.n_seq, a.T)) return;
        }
        const int ht = (a.G + RT - 1) / RT;
        const int n = KIND == LTK_ATTEND_PACKED ? min(max(a.lens[t / a.group], 0), a.cap) : a.cap;
        const int per = (n + a.splits - 1) / a.splits;
        used = (n + per - 1) / max(per, 1);
        unit = ((int64_t)t * ht + g / RT) * a.c.Hkv + h;
        at = g % RT;
    }
    if (used <= 1) return;   // written by its only split
    const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    const float* base = a.part + unit * a.splits * (int64_t)(RT * (D + 2));
    float m = kNoRef, l = 0.0f;
    at_f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = grp; s < used; s += kGroups) {
        const float* p = base + (int64_t)s * (RT * (D + 2));
        const float ms = p[RT * D + at * 2], lsum = p[RT * D + at * 2 + 1];
        const at_f32x4 x = *reinterpret_cast<const at_f32x4*>(p + at * D + 4 * lane);
        const float mn = fmaxf(m, ms), f0 = __builtin_amdgcn_exp2f(m - mn), f1 = __builtin_amdgcn_exp2f(ms - mn);
        l = l * f0 + lsum * f1;
        o = o * f0 + x * f1;
        m = mn;
    }
    *reinterpret_cast<at_f32x4*>(&s_o[grp][4 * lane]) = o;
    if (lane == 0) s_ml[grp][0] = m, s_ml[grp][1] = l;
    __syncthreads();
    if (grp != 0) return;
    float mm = kNoRef;
#pragma unroll
    for (int w = 0; w < kGroups; ++w) mm = fmaxf(mm, s_ml[w][0]);
    float sum = 0.0f;
    at_f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kGroups; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_ml[w][0] - mm);
        sum = __builtin_fmaf(f, s_ml[w][1], sum);
        const at_f32x4 x = *reinterpret_cast<const at_f32x4*>(&s_o[w][4 * lane]);
        acc = acc + x * f;
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    *reinterpret_cast<at_u32x2*>(a.out + r * D + 4 * lane) =
        at_u32x2{pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv)};
}

template <int KIND, int D, int MT>
hipError_t launch(const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    const int64_t blocks = p.units * p.splits;
    const int64_t rows = (int64_t)a.T * a.Hq;
    if (blocks > 0x7fffffff || rows > 0x7fffffff) return hipErrorInvalidValue;
    if (blocks == 0) return hipSuccess;
    if constexpr (KIND == LTK_ATTEND) {
        attend_kernel<D, MT><<<(unsigned)blocks, 64 * kWaves, finish_lds<D, MT>(), st>>>(a);
    } else {
        constexpr size_t lds = std::max(finish_lds<D, MT>(), sizeof(ListLds));
        attend_list_kernel<D, MT, KIND == LTK_ATTEND_PACKED><<<(unsigned)blocks, 64 * kWaves, lds, st>>>(a);
    }
    if (p.splits > 1) attend_join_kernel<D, MT, KIND><<<(unsigned)rows, 256, 0, st>>>(a);
    return hipGetLastError();
}

template <int KIND>
hipError_t launch_kind(int D, const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    if (D == 64) return p.mt == 1 ? launch<KIND, 64, 1>(p, a, st) : launch<KIND, 64, 2>(p, a, st);
    return p.mt == 1 ? launch<KIND, 128, 1>(p, a, st) : launch<KIND, 128, 2>(p, a, st);
}

}  // namespace

AttendPlan attend_plan(int kind, int T, int Hq, int Hkv, int D, int n_seq, int64_t entries) {
    AttendPlan p{};
    const int G = Hq / Hkv;
    if (kind == LTK_ATTEND) {
        p.mt = (int64_t)T * G > 16 * (int64_t)std::max(n_seq, 1) ? 2 : 1;   // more than 16 (row, head) pairs a sequence
        p.units = unit_bound(n_seq, T, G, 16 * p.mt, 1) * Hkv;
    } else {
        p.mt = G > 16 ? 2 : 1;
        p.units = (int64_t)T * ((G + 16 * p.mt - 1) / (16 * p.mt)) * Hkv;
    }
    // about 1,024 workgroups (four per CU), each with at least one 32-key tile per wave
    const int64_t most = std::max<int64_t>(1, (entries + kTile * kWaves - 1) / (kTile * kWaves));
    p.splits = (int)std::min<int64_t>(most, std::max<int64_t>(1, 1024 / std::max<int64_t>(p.units, 1)));
    p.ws_bytes = 256;
    if (p.splits > 1)
        p.ws_bytes = std::max<size_t>(256, (size_t)p.units * p.splits * (16 * p.mt) * (D + 2) * sizeof(float));
    return p;
}

hipError_t launch_attend(int kind, int D, const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    if (kind == LTK_ATTEND) return launch_kind<LTK_ATTEND>(D, p, a, st);
    if (kind == LTK_ATTEND_SELECTED) return launch_kind<LTK_ATTEND_SELECTED>(D, p, a, st);
    return launch_kind<LTK_ATTEND_PACKED>(D, p, a, st);
}

}  // namespace ltk
