// attend_tile.hip -- attention over the paged e4m3 cache for many rows per key
// on gfx950 (prefill chunks, packed groups): bound by the matrix cores and the
// exponentials beside them.
//
// A workgroup of four waves takes 128 (row, head) pairs of one key/value head,
// 32 a wave, and 64 keys a step.  The formulas are those of attend.hip; what
// differs is where the conversions happen.  Each key byte meets 128 rows, so
// keys and values are converted once per workgroup on their way into LDS
// (keys to bf16, values to fp16, both exact) and not in every wave:
//  - keys [64][D] bf16, read as rows of v_mfma_f32_32x32x16_bf16;
//  - values transposed, [D][64] fp16: a thread loads 4 bytes of 8 keys, pairs
//    them byte by byte and stores four 16-byte pieces, so the second product
//    reads its operand with one ds_read_b128.  The 8 keys are those whose
//    weights one lane holds after the first product, so weights go from the
//    first product's result to the second's operand in place.
// 16-byte chunks are XOR-swizzled by row so that reads of 8 rows and writes of
// 8 pieces each touch all banks.  Two stages of LDS (64 KB at D = 128), global
// loads two steps ahead, one barrier a step, two workgroups on a CU.
#include <algorithm>

#include "attend.hpp"

namespace ltk {

namespace {

typedef float at_f32x16 __attribute__((ext_vector_type(16)));
typedef int at_i32x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 128;      // (row, head) pairs of a unit
constexpr int kKeys = 64;       // keys of a step
constexpr int kThreads = 256;
constexpr int kRing = 256;      // list entries resolved together (one a thread), two such chunks in LDS
constexpr int kMinKeys = 4 * kKeys;   // least keys of a workgroup's range

__device__ __forceinline__ float max_halves(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

template <int D>
struct Stage {
    uint16_t k[kKeys * D];
    uint16_t v[D * kKeys];
    at_f32x4 scale[kKeys / 16];   // dense: c, lv, iv of each 16 keys' page
};
struct Ring {                     // listed keys, resolved
    int32_t row[2 * kRing];       // cache row of the unit's head, -1: no key
    uint32_t mask[2 * kRing];     // rows that see it
    float c[2 * kRing], lv[2 * kRing], iv[2 * kRing];
};
template <int D, bool LIST>
struct Lds {
    Stage<D> st[2];
    Ring ring[LIST ? 1 : 0];
};

// Swizzles: key rows by their low bits; value rows so that both 8 consecutive
// rows (reads) and 8 rows 4 apart (writes) get different chunks.
template <int D>
__device__ __forceinline__ int k_at(int key, int chunk) {
    return key * D + ((chunk ^ (key & 7)) << 3);
}
__device__ __forceinline__ int v_at(int d, int chunk) {
    return d * kKeys + ((chunk ^ ((d & 7) ^ ((d >> 3) & 3))) << 3);
}

// The thread's part of a step's bytes.  D = 128: every thread takes two
// 16-byte key pieces and one value patch (8 keys x 4 bytes).  D = 64: waves 2
// and 3 take the keys, waves 0 and 1 the values.
template <int D>
struct Part {
    static constexpr bool kSplit = D == 64;
    static constexpr int kPieces = D / 16;   // 16-byte pieces of a key row
    bool keys, vals;
    int key, piece;          // key pieces: rows key and key + 32
    int chunk, dq;           // value patch: 8 keys of chunk, dimensions 4 dq ..
    __device__ __forceinline__ Part() {
        const int tid = threadIdx.x;
        keys = !kSplit || tid >= 128;
        vals = !kSplit || tid < 128;
        const int i = kSplit ? (tid & 127) : tid;
        key = i / kPieces, piece = i % kPieces;
        chunk = i / (D / 4), dq = i % (D / 4);
    }
    // the patch's i-th key: its chunk holds the keys of one lane's weights
    __device__ __forceinline__ int val_key(int i) const {
        return 16 * (chunk >> 1) + 4 * (chunk & 1) + (i & 3) + ((i & 4) << 1);
    }
};
struct Raw {
    at_u32x4 k[2];
    uint32_t v[8];
};

template <int D>
__device__ __forceinline__ void store_stage(const Part<D>& p, const Raw& r, Stage<D>& s) {
    if (p.keys) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int key = p.key + 32 * x;
            *reinterpret_cast<at_bf16x8*>(s.k + k_at<D>(key, 2 * p.piece)) = bf16_of(r.k[x][0], r.k[x][1]);
            *reinterpret_cast<at_bf16x8*>(s.k + k_at<D>(key, 2 * p.piece + 1)) = bf16_of(r.k[x][2], r.k[x][3]);
        }
    }
    if (p.vals) {
        at_f16x8 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __builtin_amdgcn_perm(r.v[2 * i + 1], r.v[2 * i], 0x05010400u);
            const uint32_t hi = __builtin_amdgcn_perm(r.v[2 * i + 1], r.v[2 * i], 0x07030602u);
            const at_f16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
            const at_f16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
            const at_f16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
            const at_f16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
            o[0][2 * i] = x0[0], o[0][2 * i + 1] = x0[1];
            o[1][2 * i] = x1[0], o[1][2 * i + 1] = x1[1];
            o[2][2 * i] = x2[0], o[2][2 * i + 1] = x2[1];
            o[3][2 * i] = x3[0], o[3][2 * i + 1] = x3[1];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<at_f16x8*>(s.v + v_at(4 * p.dq + e, p.chunk)) = o[e];
    }
}

// N matrix instructions whose LDS operands are read kAhead at a time, one
// batch ahead of their use.  The scheduling barriers hold the order: left
// alone, the compiler keeps one operand and waits for LDS before every
// instruction.
constexpr int kAhead = 2;
template <int N, class V, class Read, class Use>
__device__ __forceinline__ void pipelined(Read read, Use use) {
    V f[2][kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[0][i] = read(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < N / kAhead; ++n) {
        if (n + 1 < N / kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) f[(n + 1) & 1][i] = read((n + 1) * kAhead + i);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) use(n * kAhead + i, f[n & 1][i]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Running state of a wave's 32 rows: lane (c, g) = (lane % 32, lane / 32)
// holds row c, of its accumulators the dimensions 32 t + 8 (r / 4) + 4 g + r % 4.
template <int D>
struct WaveState {
    float m, over, l;
    at_f32x16 o[D / 32];
};

// 64 keys of a stage against the wave's rows.  scale(hb, i, m, c, lv):
// constants of the lane's keys 4 i .. 4 i + 3 of half hb (i < 4), lv less m;
// scale.inverse: their 1 / vs; mask(hb, y): hides keys the lane's row does not
// see.
template <int D, class Scale, class Mask>
__device__ __forceinline__ void step_keys(const Stage<D>& s, const at_bf16x8 (&q)[D / 16], WaveState<D>& st, Scale scale,
                                          Mask mask) {
    const int lane = threadIdx.x & 63, c = lane & 31, g = lane >> 5;
    at_f32x16 x[2];
#pragma unroll
    for (int r = 0; r < 16; ++r) x[0][r] = x[1][r] = 0.0f;
    pipelined<D / 8, at_bf16x8>(   // n = 2 j + hb
        [&](int n) { return *reinterpret_cast<const at_bf16x8*>(s.k + k_at<D>(32 * (n & 1) + c, (n & ~1) + g)); },
        [&](int n, const at_bf16x8& kf) {
            x[n & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[n >> 1], x[n & 1], 0, 0, 0);
        });
    // scores relative to the reference
    float top = -INFINITY;
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            at_f32x4 cc, lv;
            scale(hb, i, st.m, cc, lv);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[hb][4 * i + r] = __builtin_fmaf(x[hb][4 * i + r], cc[r], lv[r]);
        }
        mask(hb, x[hb]);
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, x[hb][r]);
    }
    if (__any(top > st.over)) {
        const float up = max_halves(top);
        const bool move = up > st.over;
        const float d = move ? up : 0.0f;
        const float f = st.over == kSlack ? __builtin_amdgcn_exp2f(-d) : 1.0f;   // (nothing to scale at the first move)
        st.m += d;
        st.over = move ? kSlack : st.over;
        st.l *= f;
#pragma unroll
        for (int t = 0; t < D / 32; ++t) st.o[t] *= f;
#pragma unroll
        for (int r = 0; r < 16; ++r) x[0][r] -= d, x[1][r] -= d;
    }
    at_f16x8 p[4];
#pragma unroll
    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            at_f32x4 iv;
            scale.inverse(hb, i, iv);
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
                const float p0 = __builtin_amdgcn_exp2f(x[hb][4 * i + r]);
                const float p1 = __builtin_amdgcn_exp2f(x[hb][4 * i + r + 1]);
                st.l = __builtin_fmaf(p0, iv[r], st.l);
                st.l = __builtin_fmaf(p1, iv[r + 1], st.l);
                const at_f32x2 pp{p0, p1};
                const at_f16x2 ph = __builtin_convertvector(pp, at_f16x2);
                p[2 * hb + (i >> 1)][4 * (i & 1) + r] = ph[0];
                p[2 * hb + (i >> 1)][4 * (i & 1) + r + 1] = ph[1];
            }
        }
    pipelined<D / 8, at_f16x8>(    // n = (D / 32) w + t
        [&](int n) {
            const int w = n / (D / 32), t = n % (D / 32);
            return *reinterpret_cast<const at_f16x8*>(s.v + v_at(32 * t + c, 2 * w + g));
        },
        [&](int n, const at_f16x8& vf) {
            const int w = n / (D / 32), t = n % (D / 32);
            st.o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, p[w], st.o[t], 0, 0, 0);
        });
}

// The unit's rows, flattened (row, head) from f0 to f1: row r0 + f / G, head
// h G + f % G.
struct UnitRows {
    int r0, f0, f1, h;
};
__device__ __forceinline__ int64_t out_row(const AttendArgs& a, const UnitRows& u, int f) {
    if (f >= u.f1) return -1;
    const int i = f / a.G;
    return (int64_t)(u.r0 + i) * a.Hq + u.h * a.G + (f - i * a.G);
}

template <int D>
__device__ __forceinline__ void begin_rows(const AttendArgs& a, int64_t row, at_bf16x8 (&q)[D / 16], WaveState<D>& st) {
    const int g = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        at_u32x4 w{0u, 0u, 0u, 0u};
        if (row >= 0) w = *reinterpret_cast<const at_u32x4*>(a.q + row * D + 16 * j + 8 * g);
        q[j] = __builtin_bit_cast(at_bf16x8, w);
    }
    st.m = 0.0f;
    st.over = -INFINITY;
    st.l = 0.0f;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) st.o[t][r] = 0.0f;
}

// Rows written as bf16 where the workgroup saw all of their keys (part ==
// NULL), else as a part: [kRows][D] floats, then [kRows] (m, l).
template <int D>
constexpr int part_floats() {
    return kRows * (D + 2);
}
template <int D>
__device__ __forceinline__ void end_rows(const AttendArgs& a, int64_t row, const WaveState<D>& st, float* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 31, g = lane >> 5;
    const float l = sum_halves(st.l);
    if (row < 0) return;
    if (!part) {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        uint16_t* dst = a.out + row * D;
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<at_u32x2*>(dst + 32 * t + 8 * i + 4 * g) =
                    at_u32x2{pack_bf16(st.o[t][4 * i] * inv, st.o[t][4 * i + 1] * inv),
                             pack_bf16(st.o[t][4 * i + 2] * inv, st.o[t][4 * i + 3] * inv)};
        return;
    }
    const int r = 32 * wave + c;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<at_f32x4*>(part + (size_t)r * D + 32 * t + 8 * i + 4 * g) =
                at_f32x4{st.o[t][4 * i], st.o[t][4 * i + 1], st.o[t][4 * i + 2], st.o[t][4 * i + 3]};
    if (g == 0) {
        part[(size_t)kRows * D + 2 * r] = l > 0.0f ? st.m : kNoRef;
        part[(size_t)kRows * D + 2 * r + 1] = l;
    }
}

// ------------------------------------------------------------ dense keys

// Work is cut evenly as in attend.hip, here on a line of keys: the unit of
// row tile i counts A + i Q keys, at least as many as its last row sees, so
// that a sequence's prefix sums have a closed form.
struct SeqLine {
    SeqRows sr;
    int tiles;       // row tiles
    int64_t A, Q;
    __device__ __forceinline__ int64_t cost(int i) const { return A + i * Q; }
    __device__ __forceinline__ int64_t before(int i) const { return i * A + Q * ((int64_t)i * (i - 1) / 2); }
};
__device__ __forceinline__ SeqLine seq_line(const AttendArgs& a, int b) {
    SeqLine s;
    s.sr = seq_rows(a.bt, b, a.T);
    const int n = s.sr.r1 - s.sr.r0;
    s.tiles = (int)(((int64_t)n * a.G + kRows - 1) / kRows);
    s.Q = uniform((kRows + a.G - 1) / a.G);
    const int64_t cap = (int64_t)a.bt.max_pages << a.c.page_shift;
    s.A = max(min((int64_t)s.sr.pos0 + 1 + s.Q, cap), (int64_t)1);
    // a window's rows see at most the sinks, the window and the tiles' borders
    const int64_t win = (int64_t)a.n_sink + a.window + s.Q + 1 + 3 * kKeys;
    if (a.window > 0 && win < s.A) s.A = win, s.Q = 0;
    return s;
}

// Key tiles of rows at positions pos_lo .. pos_hi, as in attend.hip.
struct KeyTiles {
    int lo, hi, sink_tiles, win_tile0, tiles;
};
__device__ __forceinline__ KeyTiles key_tiles(const AttendArgs& a, int pos_lo, int pos_hi) {
    KeyTiles k;
    k.hi = min(max(pos_hi + 1, 0), a.bt.max_pages << a.c.page_shift);
    k.lo = a.window > 0 ? min(max(max(pos_lo, 0) - a.window + 1, 0), k.hi) : 0;
    k.sink_tiles = a.window > 0 ? (min(a.n_sink, k.lo) + kKeys - 1) / kKeys : 0;
    k.win_tile0 = max(k.lo / kKeys, k.sink_tiles);
    k.tiles = k.sink_tiles + max((k.hi + kKeys - 1) / kKeys - k.win_tile0, 0);
    return k;
}

struct DenseScale {
    const at_f32x4* s;   // the stage's four pages: c, lv, iv
    __device__ __forceinline__ void operator()(int hb, int i, float m, at_f32x4& c, at_f32x4& lv) const {
        const at_f32x4 x = s[2 * hb + (i >> 1)];
        const float y = x[1] - m;
        c = at_f32x4{x[0], x[0], x[0], x[0]};
        lv = at_f32x4{y, y, y, y};
    }
    __device__ __forceinline__ void inverse(int hb, int i, at_f32x4& iv) const {
        const float x = s[2 * hb + (i >> 1)][2];
        iv = at_f32x4{x, x, x, x};
    }
};

template <int D>
__device__ __forceinline__ void dense_unit(const AttendArgs& a, const SeqRows& sr, int b, const UnitRows& u,
                                           const KeyTiles& kt, int t0, int t1, Lds<D, false>& ls, float* part) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, g = lane >> 5;
    const int fw = u.f0 + 32 * wave;                      // the wave's rows [fw, fw1)
    const int fw1 = min(fw + 32, u.f1);
    const int pos_lo = sr.pos0 + uniform(fw / a.G), pos_hi = sr.pos0 + uniform((max(fw1, 1) - 1) / a.G);
    const int64_t row = out_row(a, u, fw + c);
    const int pos = row < 0 ? -1 : sr.pos0 + (fw + c) / a.G;
    const int from = a.window > 0 ? max(pos, 0) - a.window : -1;   // the lane's row sees keys behind it, and the sinks
    at_bf16x8 q[D / 16];
    WaveState<D> st;
    begin_rows<D>(a, row, q, st);

    const int32_t* table = a.bt.table + (size_t)b * a.bt.max_pages;
    const int page = 1 << a.c.page_shift;
    const Part<D> p;
    auto key0_of = [&](int t) { return (t < kt.sink_tiles ? t : kt.win_tile0 + t - kt.sink_tiles) * kKeys; };
    // pages of a step's four 16-key groups; a lane holds one of the next 16 steps'
    // (named, not an array: an array copied from step to step stays in scratch
    // memory, and the wait for it is a wait for every load in flight)
    struct Ids {
        int p0, p1, p2, p3;
        __device__ __forceinline__ int get(int i) const { return i == 0 ? p0 : i == 1 ? p1 : i == 2 ? p2 : p3; }
        __device__ __forceinline__ bool all() const { return (p0 | p1 | p2 | p3) >= 0; }
    };
    PageLanes pl;
    auto lane_key = [&](int block) {
        const int t = t0 + 16 * block + (lane >> 2);
        return t < t1 ? key0_of(t) + 16 * (lane & 3) : -1;
    };
    // (a page with no visible key is not looked at: its scale and bytes may be anything)
    auto seen = [&](int key) { return (key < kt.hi) & ((key + 15 >= kt.lo) | (key < a.n_sink)); };
    auto cache_row = [&](const Ids& x, int key0, int grp, int key) -> size_t {   // grp: key / 16 of the step
        return (((size_t)max(x.get(grp), 0) * a.c.Hkv + u.h) << a.c.page_shift) + ((key0 + key) & (page - 1));
    };
    Raw raw;
    auto load = [&](int t, Ids& x) {
        const int n = t - t0, key0 = key0_of(t);
        if (n % 16 == 0) pl.turn(table, a, u.h, n / 16, lane_key, seen);
        const int at = 4 * (n % 16);
        x = Ids{pl.page(at), pl.page(at + 1), pl.page(at + 2), pl.page(at + 3)};
        if (p.keys) {
#pragma unroll
            for (int y = 0; y < 2; ++y)
                raw.k[y] = *reinterpret_cast<const at_u32x4*>(
                    a.c.k + cache_row(x, key0, (p.key + 32 * y) >> 4, p.key + 32 * y) * D + 16 * p.piece);
        }
        if (p.vals) {
            const uint8_t* v = a.c.v + cache_row(x, key0, p.chunk >> 1, p.val_key(0)) * D + 4 * p.dq;
#pragma unroll
            for (int i = 0; i < 8; ++i) raw.v[i] = *reinterpret_cast<const uint32_t*>(v + (p.val_key(i) - p.val_key(0)) * D);
        }
    };
    auto seen_by_all = [&](int key0, const Ids& x, int lo, int hi) {   // every key of the step by rows at lo .. hi
        return x.all() && key0 + kKeys - 1 <= lo &&
               key0 + kKeys <= kt.hi && (a.window <= 0 || key0 > hi - a.window || key0 + kKeys <= a.n_sink);
    };
    auto store = [&](int t, const Ids& x, Stage<D>& s) {
        const int key0 = key0_of(t);
        const bool clean = x.all() && key0 + kKeys <= kt.hi &&
                           (key0 >= kt.lo || key0 + kKeys <= a.n_sink);
        if (!clean) {
            // bytes of keys that no row sees may be NaN: their weights are 0, so the values must be finite
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int key = key0 + p.val_key(i);
                const bool ok = (x.get(p.chunk >> 1) >= 0) & (key < kt.hi) & ((key >= kt.lo) | (key < a.n_sink));
                raw.v[i] = ok ? raw.v[i] : 0u;
            }
        }
        store_stage<D>(p, raw, s);
        const int n = t - t0;
        if (wave == 0) {   // (before the loads of step t + 1, which may turn the lanes)
            if (n % 16 == 0) pl.scales(a.c2);
            if ((lane >> 2) == n % 16) s.scale[lane & 3] = at_f32x4{pl.s.c_, pl.s.lv_, pl.s.iv_, 0.0f};
        }
    };
    auto step = [&](int t, const Ids& x, const Stage<D>& s) {
        const int key0 = key0_of(t);
        if (fw >= fw1 || key0 > pos_hi) return;   // no row of the wave sees a key of it
        if (a.window > 0 && key0 + kKeys - 1 <= max(pos_lo, 0) - a.window && key0 >= a.n_sink) return;
        const bool all = seen_by_all(key0, x, pos_lo, pos_hi);
        step_keys<D>(s, q, st, DenseScale{s.scale}, [&](int hb, at_f32x16& y) {
            if (all) return;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int key = key0 + 32 * hb + 8 * (r >> 2) + 4 * g + (r & 3);
                const bool ok = (x.get(2 * hb + (r >> 3)) >= 0) & (key <= pos) & (key < kt.hi) &
                                ((key > from) | (key < a.n_sink));
                y[r] = ok ? y[r] : -INFINITY;
            }
        });
    };

    // step t computes from one stage while t + 1 is written to the other and
    // t + 2 is on its way
    if (t0 < t1) {
        Ids now, next, far;
        pl.read(table, a, 0, lane_key);
        load(t0, now);
        store(t0, now, ls.st[0]);
        next = far = now;
        if (t0 + 1 < t1) load(t0 + 1, next);
        __syncthreads();
        for (int t = t0; t < t1; ++t) {
            const int x = (t - t0) & 1;
            if (t + 1 < t1) store(t + 1, next, ls.st[x ^ 1]);
            if (t + 2 < t1) load(t + 2, far);
            step(t, now, ls.st[x]);
            now = next;
            next = far;
            __syncthreads();
        }
    }
    end_rows<D>(a, row, st, part);
}

// What a workgroup leaves to join, in the workspace: the unit that began in
// its range and goes on in those behind it.  Its parts are the workgroup's
// (slot), then the first ones of the n - 1 workgroups that follow.
struct Crossing {
    int n, slot;   // n == 0: none
    UnitRows u;
};
struct ScanLds {
    int64_t wave[kThreads / 64];
    int64_t at;   // place of sequence b, which the workgroup's range begins in
    int b;
};
__device__ __forceinline__ int64_t scan_256(int64_t x, ScanLds& ls, int64_t& sum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 63) ls.wave[wave] = x;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wave) x += ls.wave[w];
        sum += ls.wave[w];
    }
    return x;
}
__device__ __forceinline__ int64_t line_of(const AttendArgs& a, int b) {
    if (b >= a.bt.n_seq) return 0;
    const SeqLine s = seq_line(a, b);
    return s.before(s.tiles) * a.c.Hkv;
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void attend_tile_kernel(AttendArgs a) {
    extern __shared__ at_u32x4 sh[];
    Lds<D, false>& ls = *reinterpret_cast<Lds<D, false>*>(sh);
    __shared__ ScanLds sc;
    int64_t total = 0, sum;
    for (int b0 = 0; b0 < a.bt.n_seq; b0 += kThreads) {
        scan_256(line_of(a, b0 + threadIdx.x), sc, sum);
        total += uniform(sum);
    }
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kMinKeys);
    // Workgroups go to the eight XCDs in turn: each XCD takes a stretch of the
    // line, so that the row tiles of one head read its keys through one L2.
    const int n8 = gridDim.x / 8;
    const int me = (int)blockIdx.x < 8 * n8 ? (blockIdx.x % 8) * n8 + blockIdx.x / 8 : (int)blockIdx.x;
    int64_t at = me * per;
    const int64_t end = min(at + per, total);
    Crossing* crossing = reinterpret_cast<Crossing*>(a.head) + me;
    if (threadIdx.x == 0) crossing->n = 0;
    if (at >= end) return;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.bt.n_seq; b0 += kThreads) {
        const int64_t w = line_of(a, b0 + threadIdx.x), x = before + scan_256(w, sc, sum);
        if (x - w <= at && at < x) sc.b = b0 + threadIdx.x, sc.at = x - w;
        before += uniform(sum);
        if (at < before) break;
    }
    __syncthreads();
    int b = uniform(sc.b);
    int64_t first = uniform(sc.at);
    SeqLine s = seq_line(a, b);
    while (true) {
        const int64_t per_head = s.before(s.tiles);
        int h = uniform((int)((at - first) / per_head));
        const int64_t off = at - first - h * per_head;
        int i = 0, hi = s.tiles - 1;   // the row tile that holds off
        while (i < hi) {
            const int mid = (i + hi + 1) >> 1;
            if (s.before(mid) <= off)
                i = mid;
            else
                hi = mid - 1;
        }
        for (; h < a.c.Hkv && at < end; ++h, i = 0)
            for (; i < s.tiles && at < end; ++i) {
                const int64_t us = first + h * per_head + s.before(i), cost = s.cost(i);
                UnitRows u;
                u.r0 = s.sr.r0;
                u.h = h;
                u.f0 = i * kRows;
                u.f1 = min(u.f0 + kRows, (s.sr.r1 - s.sr.r0) * a.G);
                const KeyTiles kt = key_tiles(a, s.sr.pos0 + uniform(u.f0 / a.G), s.sr.pos0 + uniform((u.f1 - 1) / a.G));
                // a step belongs to the range that its first key lies in
                const int64_t k0 = at - us, k1 = min(end - us, cost);
                const int t0 = (int)((k0 + kKeys - 1) / kKeys), t1 = (int)((k1 + kKeys - 1) / kKeys);
                const bool whole = k0 == 0 && k1 == cost;
                float* part = whole ? nullptr : a.part + (2 * (int64_t)me + (at == me * per ? 0 : 1)) * part_floats<D>();
                dense_unit<D>(a, s.sr, b, u, kt, t0, min(t1, kt.tiles), ls, part);
                if (k0 == 0 && k1 < cost && threadIdx.x == 0)
                    *crossing = Crossing{(int)((us + cost - 1) / per) - me + 1, 2 * me + (at == me * per ? 0 : 1), u};
                at = us + k1;
            }
        if (at >= end) return;
        first += a.c.Hkv * per_head;
        do s = seq_line(a, ++b);
        while (s.tiles == 0);
    }
}

// ------------------------------------------------------------ packed lists

struct ListScale {
    const Ring* r;
    int at, g;   // the step's place in the ring, the lane's half
    __device__ __forceinline__ int key(int hb, int i) const { return at + 32 * hb + 8 * i + 4 * g; }
    __device__ __forceinline__ void operator()(int hb, int i, float m, at_f32x4& c, at_f32x4& lv) const {
        c = *reinterpret_cast<const at_f32x4*>(r->c + key(hb, i));
        lv = *reinterpret_cast<const at_f32x4*>(r->lv + key(hb, i));
        lv = at_f32x4{lv[0] - m, lv[1] - m, lv[2] - m, lv[3] - m};
    }
    __device__ __forceinline__ void inverse(int hb, int i, at_f32x4& iv) const {
        iv = *reinterpret_cast<const at_f32x4*>(r->iv + key(hb, i));
    }
};

// A unit is 128 (row, head) pairs of one group and key/value head; its keys
// are the group's list, cut into a.splits.
template <int D>
__global__ __launch_bounds__(kThreads, 2) void attend_tile_list_kernel(AttendArgs a) {
    extern __shared__ at_u32x4 sh[];
    Lds<D, true>& ls = *reinterpret_cast<Lds<D, true>*>(sh);
    Ring& ring = ls.ring[0];
    const int ht = (a.group * a.G + kRows - 1) / kRows;   // row tiles of a group
    UnitRows u;
    u.h = uniform((int)(blockIdx.x % a.c.Hkv));
    int rest = uniform((int)(blockIdx.x / a.c.Hkv));
    const int tile = uniform(rest % ht);
    rest = uniform(rest / ht);
    const int split = uniform(rest % a.splits), grp = uniform(rest / a.splits);
    u.r0 = grp * a.group;
    u.f0 = tile * kRows;
    u.f1 = min(u.f0 + kRows, min(a.group, a.T - u.r0) * a.G);
    if (u.f0 >= u.f1) return;
    const int n = min(max(a.lens[grp], 0), a.cap);
    const int per = uniform(((n + kKeys - 1) / kKeys + a.splits - 1) / a.splits * kKeys);
    const int e0 = split * per, e1 = min(e0 + per, n);
    if (split > 0 && e0 >= e1) return;
    const int used = per > 0 ? (n + per - 1) / per : 1;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, g = lane >> 5;
    const int fw = u.f0 + 32 * wave;
    const int64_t row = out_row(a, u, fw + c);
    const int pos0 = max(a.bt.len[0], 0) - a.T;
    const int qi = row < 0 ? 0 : (fw + c) / a.G;             // the lane's row in its group
    const int last = pos0 + u.r0 + (u.f1 - 1) / a.G;          // the unit's last row
    const int end = min(max(last + 1, 0), a.bt.max_pages << a.c.page_shift);
    at_bf16x8 q[D / 16];
    WaveState<D> st;
    begin_rows<D>(a, row, q, st);

    const int32_t* list = a.list + (size_t)grp * a.cap;
    const uint32_t* masks = a.masks + (size_t)grp * a.cap;
    const int page = 1 << a.c.page_shift;
    // Rows of the group at or after a key's position may see it: a key after
    // some of the group's rows loses their bits.
    struct Entry {
        int s, pid;
        uint32_t mask;
        float ks, vs;
    } en;
    auto entry_load = [&](int chunk) {
        const int e = e0 + chunk * kRing + tid;
        en.s = -1, en.mask = 0u;
        if (e < e1) en.s = list[e], en.mask = masks[e];
    };
    auto entry_page = [&]() {
        en.pid = -1;
        if (en.s >= 0 && en.s < end) en.pid = a.bt.table[en.s >> a.c.page_shift];
        if (en.pid >= a.c.n_pages) en.pid = -1;
    };
    auto entry_scale = [&]() {
        const size_t at = (size_t)max(en.pid, 0) * a.c.Hkv + u.h;
        en.ks = en.pid >= 0 ? a.c.ks[at] : 1.0f;
        en.vs = en.pid >= 0 ? a.c.vs[at] : 1.0f;
    };
    auto entry_store = [&](int chunk) {
        const int at = (chunk & 1) * kRing + tid;
        const int later = en.pid >= 0 ? en.s - (pos0 + u.r0) : 0;   // rows of the group before the key
        uint32_t m = en.pid >= 0 ? en.mask : 0u;
        if (later > 0) m &= later < 32 ? ~0u << later : 0u;
        const PageScale ps = page_scale(a.c2, en.ks, en.vs);
        ring.row[at] = en.pid >= 0 ? (int)((((size_t)en.pid * a.c.Hkv + u.h) << a.c.page_shift) + (en.s & (page - 1))) : -1;
        ring.mask[at] = m;
        ring.c[at] = ps.c_, ring.lv[at] = ps.lv_, ring.iv[at] = ps.iv_;
    };
    const Part<D> p;
    Raw raw;
    uint32_t none = 0;   // bit i: the patch's i-th key is no key
    auto load = [&](int t) {
        const int at = (t * kKeys) & (2 * kRing - 1);
        if (p.keys) {
#pragma unroll
            for (int y = 0; y < 2; ++y)
                raw.k[y] = *reinterpret_cast<const at_u32x4*>(a.c.k + (size_t)max(ring.row[at + p.key + 32 * y], 0) * D +
                                                              16 * p.piece);
        }
        if (p.vals) {
            const at_i32x4 r0 = *reinterpret_cast<const at_i32x4*>(ring.row + at + p.val_key(0));
            const at_i32x4 r1 = *reinterpret_cast<const at_i32x4*>(ring.row + at + p.val_key(4));
            none = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i < 4 ? r0[i & 3] : r1[i & 3];
                none |= r < 0 ? 1u << i : 0u;
                raw.v[i] = *reinterpret_cast<const uint32_t*>(a.c.v + (size_t)max(r, 0) * D + 4 * p.dq);
            }
        }
    };
    auto store = [&](Stage<D>& s) {
        if (__any(none != 0)) {   // bytes behind no key may be NaN
#pragma unroll
            for (int i = 0; i < 8; ++i) raw.v[i] = (none >> i) & 1u ? 0u : raw.v[i];
        }
        store_stage<D>(p, raw, s);
    };
    auto step = [&](int t, const Stage<D>& s) {
        if (fw >= u.f1) return;
        const int at = (t * kKeys) & (2 * kRing - 1);
        step_keys<D>(s, q, st, ListScale{&ring, at, g}, [&](int hb, at_f32x16& y) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const at_i32x4 m = *reinterpret_cast<const at_i32x4*>(ring.mask + at + 32 * hb + 8 * i + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // the row's bit over the whole word selects the score or -inf
                    const uint32_t see = (uint32_t)__builtin_amdgcn_sbfe(m[r], qi, 1);
                    y[4 * i + r] = __uint_as_float((see & __float_as_uint(y[4 * i + r])) | (~see & 0xff800000u));
                }
            }
        });
    };

    const int steps = (e1 - e0 + kKeys - 1) / kKeys;
    constexpr int kPer = kRing / kKeys;   // steps of a chunk
    if (steps > 0) {
        entry_load(0);
        entry_page();
        entry_scale();
        entry_store(0);
        entry_load(1);
        __syncthreads();
        load(0);
        store(ls.st[0]);
        if (steps > 1) load(1);
        __syncthreads();
        // a chunk's entries are read in the last two steps of the chunk two
        // before it, and resolved in the first two of the one before it
        for (int t = 0; t < steps; ++t) {
            const int x = t & 1, ph = t % kPer, chunk = t / kPer;
            if (t + 1 < steps) store(ls.st[x ^ 1]);
            if (t + 2 < steps) load(t + 2);
            if (ph == 0) entry_page();
            step(t, ls.st[x]);
            if (ph == 0) entry_scale();
            if (ph == 1) entry_store(chunk + 1);
            if (ph == 2) entry_load(chunk + 2);
            __syncthreads();
        }
    }
    const int64_t slot = (((int64_t)grp * ht + tile) * a.c.Hkv + u.h) * a.splits + split;
    end_rows<D>(a, row, st, used > 1 ? a.part + slot * part_floats<D>() : nullptr);
}

// ------------------------------------------------------- joining the parts

// Sum of n parts of one row by D / 4 lanes: part i at slot0 (i == 0) or
// slot1 + (i - 1) step.
template <int D>
__device__ __forceinline__ void join_row(const AttendArgs& a, int64_t row, int at, int n, int64_t slot0, int64_t slot1,
                                         int step) {
    const int lane = threadIdx.x % (D / 4);
    float m = kNoRef, l = 0.0f;
    at_f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float* p = a.part + (i == 0 ? slot0 : slot1 + (int64_t)(i - 1) * step) * part_floats<D>();
        const float mi = p[kRows * D + at * 2], li = p[kRows * D + at * 2 + 1];
        const at_f32x4 x = *reinterpret_cast<const at_f32x4*>(p + at * D + 4 * lane);
        const float mn = fmaxf(m, mi), f0 = __builtin_amdgcn_exp2f(m - mn), f1 = __builtin_amdgcn_exp2f(mi - mn);
        l = l * f0 + li * f1;
        o = o * f0 + x * f1;
        m = mn;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    *reinterpret_cast<at_u32x2*>(a.out + row * D + 4 * lane) =
        at_u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
}

constexpr int kJoinRows = 8;   // rows of a joining workgroup

template <int D>
__global__ __launch_bounds__(kJoinRows * D / 4) void attend_tile_join_kernel(AttendArgs a) {
    const Crossing x = reinterpret_cast<const Crossing*>(a.head)[blockIdx.x];
    const int at = blockIdx.y * kJoinRows + threadIdx.x / (D / 4);
    const int64_t row = x.n > 0 ? out_row(a, x.u, x.u.f0 + at) : -1;
    if (row >= 0) join_row<D>(a, row, at, x.n, x.slot, 2 * ((int64_t)blockIdx.x + 1), 2);
}

template <int D>
__global__ __launch_bounds__(kJoinRows * D / 4) void attend_tile_list_join_kernel(AttendArgs a) {
    const int64_t r = (int64_t)blockIdx.x * kJoinRows + threadIdx.x / (D / 4);   // row * Hq + head
    if (r >= (int64_t)a.T * a.Hq) return;
    const int t = (int)(r / a.Hq), head = (int)(r % a.Hq), h = head / a.G;
    const int grp = t / a.group, ht = (a.group * a.G + kRows - 1) / kRows;
    const int n = min(max(a.lens[grp], 0), a.cap);
    const int per = ((n + kKeys - 1) / kKeys + a.splits - 1) / a.splits * kKeys;
    const int used = per > 0 ? (n + per - 1) / per : 1;
    if (used <= 1) return;
    const int f = (t % a.group) * a.G + (head - h * a.G);
    const int64_t slot0 = (((int64_t)grp * ht + f / kRows) * a.c.Hkv + h) * a.splits;
    join_row<D>(a, r, f % kRows, used, slot0, slot0 + 1, 1);
}

template <int D, bool LIST>
hipError_t launch_d(const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    constexpr size_t lds = sizeof(Lds<D, LIST>);
    const void* fn = LIST ? reinterpret_cast<const void*>(attend_tile_list_kernel<D>)
                          : reinterpret_cast<const void*>(attend_tile_kernel<D>);
    if (lds > 65536)
        (void)hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if constexpr (LIST)
        attend_tile_list_kernel<D><<<(unsigned)p.blocks, kThreads, lds, st>>>(a);
    else
        attend_tile_kernel<D><<<(unsigned)p.blocks, kThreads, lds, st>>>(a);
    constexpr int threads = kJoinRows * D / 4;
    if (p.join && LIST)
        attend_tile_list_join_kernel<D>
            <<<(unsigned)(((int64_t)a.T * a.Hq + kJoinRows - 1) / kJoinRows), threads, 0, st>>>(a);
    else if (p.join)
        attend_tile_join_kernel<D><<<dim3((unsigned)p.blocks, kRows / kJoinRows), threads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

AttendPlan attend_tile_plan(int kind, int T, int Hq, int Hkv, int D, int n_seq, int64_t entries, int group) {
    AttendPlan p{};
    p.tile = true;
    const int G = Hq / Hkv;
    const size_t part = (size_t)kRows * (D + 2) * sizeof(float);
    if (kind == LTK_ATTEND) {
        const int64_t units = ((int64_t)T * G / kRows + n_seq) * Hkv;
        const int64_t most = (units * (entries + kKeys) + kMinKeys - 1) / kMinKeys;
        p.blocks = std::max<int64_t>(1, std::min<int64_t>(most, 512));   // two a CU
        p.join = p.blocks > 1;
        p.head_bytes = (sizeof(Crossing) * (size_t)p.blocks + 255) / 256 * 256;
        p.ws_bytes = p.head_bytes + (p.join ? (size_t)p.blocks * 2 * part : 0);
        return p;
    }
    const int64_t units = (int64_t)((T + group - 1) / group) * ((group * G + kRows - 1) / kRows) * Hkv;
    const int64_t most = (entries + kKeys - 1) / kKeys;
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(most, 512 / std::max<int64_t>(units, 1)));
    p.blocks = units * p.splits;
    p.join = p.splits > 1;
    p.ws_bytes = std::max<size_t>(256, p.join ? (size_t)p.blocks * part : 0);
    return p;
}

hipError_t launch_attend_tile(int kind, int D, const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    if (p.blocks > 0x7fffffff) return hipErrorInvalidValue;
    if (kind == LTK_ATTEND) return D == 64 ? launch_d<64, false>(p, a, st) : launch_d<128, false>(p, a, st);
    return D == 64 ? launch_d<64, true>(p, a, st) : launch_d<128, true>(p, a, st);
}

}  // namespace ltk
