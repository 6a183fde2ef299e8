// attend.hip -- attention over the paged e4m3 cache for few rows per key on
// gfx950 (decode, speculative decode, selected keys, packed groups of few
// rows): bound by reading the cache once.
//
// For a query row q and the keys s it sees, with page scales ks and vs,
//   y_s = scale log2(e) ks (q . k_s) + log2(vs)
//   out = sum_s 2^(y_s - m) vbyte_s / sum_s 2^(y_s - m) / vs,
// one pass with a running reference m: moving the value scale into the
// exponent keeps the weights 2^(y - m) within fp16 whatever the scales are,
// and the divisor takes it out again (for scales below kSmallScale by an
// exponential of its own).
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
// 8, so most tiles need no exchange between lanes; the weights' sums of the
// four lane groups are joined once at the end.
//
// Two tiles a wave, one in use and one on its way: 8 KB a tile at D = 128, and
// with two waves a SIMD 64 KB a CU on their way, which covers the latency of
// memory.  64 decoding sequences of up to 16,384 tokens (64 heads on 8, D = 128,
// 1.11 GB of cache) take 202 us, 5.5 TB/s (a copy reaches 5.0, reads alone 6.4);
// the join adds 5.  Eight rows over 1,048,576 tokens (2.15 GB) take 495 to 540 us, 4.0 to
// 4.3 TB/s: each byte is converted for two units of 32 rows, and conversions,
// exponentials and matrix instructions fill the issue slots.  145 rows on lists
// of 2,048 keys each (four key/value heads) take 54 us, 4.9 TB/s of the lists'
// keys.  The smallest calls
// (one row, 4,096 tokens) take 6.6 us and 3.9 for the join: launches and the
// chain length, page id, keys, values.
#include <algorithm>

#include "attend_join.hpp"

namespace ltk {

namespace {

constexpr int kWaves = 4;            // (256 threads: AttendPlan::fits)
constexpr int kTile = 32;            // keys per wave step
constexpr int kMinPer = 2 * kWaves;  // least key tiles of a workgroup's range: two per wave
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

// The wave's share of 32 keys: halves A (keys 0..15) and B (16..31).
template <int D>
struct KvTile {
    at_u32x4 k[2][D / 64];          // key row c of each half, bytes 64 h + 16 g
    uint32_t v[8][D / 64];          // the lane's 8 keys, bytes c D/16 ..
};

struct KeyScale {   // listed keys: one set each
    at_f32x4 c_, lv_, iv_;   // the lane's keys 4 g + i
    __device__ __forceinline__ float c(int i) const { return c_[i]; }
    __device__ __forceinline__ float lv(int i) const { return lv_[i]; }
    __device__ __forceinline__ float iv(int i) const { return iv_[i]; }
};

// Running state of 16 query rows: reference, weight sum (of the lane's keys)
// and the D / 16 x 4 accumulators of row c, dimensions (4 g + r) D/16 + e.
template <int D>
struct RowState {
    float m, over, l;
    at_f32x4 o[D / 16];
};

// Word w of the lane's value bytes as matrix operands: operand e holds byte
// 4 w + e of its 8 keys.
template <int D>
__device__ __forceinline__ void value_operands(const KvTile<D>& t, int w, at_f16x8 (&a)[4]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {   // key pair (2p, 2p + 1)
        const uint32_t lo = __builtin_amdgcn_perm(t.v[2 * p + 1][w], t.v[2 * p][w], 0x05010400u);
        const uint32_t hi = __builtin_amdgcn_perm(t.v[2 * p + 1][w], t.v[2 * p][w], 0x07030602u);
        const at_f16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
        const at_f16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
        const at_f16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
        const at_f16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
        a[0][2 * p] = x0[0], a[0][2 * p + 1] = x0[1];
        a[1][2 * p] = x1[0], a[1][2 * p + 1] = x1[1];
        a[2][2 * p] = x2[0], a[2][2 * p + 1] = x2[1];
        a[3][2 * p] = x3[0], a[3][2 * p + 1] = x3[1];
    }
}

// One 32-key tile against MT x 16 query rows.  query(mt, j) is operand j of
// row tile mt; mask(mt, a, i) says whether the lane's row of tile mt sees key
// 16 a + 4 g + i of the tile, asked only where `masked` (the same in all lanes).
// `small`, not 0: the tile may hold keys of small value scales (the same in all lanes).
//
// The scheduling barriers keep the parts apart: left alone, the compiler
// converts all of a tile's bytes first and holds 64 registers of operands.
template <int D, int MT, class Query, class Scale, class Mask>
__device__ __forceinline__ void tile_step(const KvTile<D>& t, Query query, const Scale (&hs)[2], RowState<D> (&st)[MT],
                                          bool masked, uint32_t small, Mask mask) {
    at_f32x4 s[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) s[mt][0] = s[mt][1] = at_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const at_bf16x8 k0 = bf16_of(t.k[0][j / 2][2 * (j % 2)], t.k[0][j / 2][2 * (j % 2) + 1]);
        const at_bf16x8 k1 = bf16_of(t.k[1][j / 2][2 * (j % 2)], t.k[1][j / 2][2 * (j % 2) + 1]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const at_bf16x8 qf = query(mt, j);
            s[mt][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf, s[mt][0], 0, 0, 0);
            s[mt][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf, s[mt][1], 0, 0, 0);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    at_f16x8 p[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float y[8], top = -INFINITY;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[4 * a + i] = __builtin_fmaf(s[mt][a][i], hs[a].c(i), hs[a].lv(i) - st[mt].m);
        if (masked) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[4 * a + i] = mask(mt, a, i) ? y[4 * a + i] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, y[i]);
        if ((__ballot(top > st[mt].over) | small) != 0) {   // (one branch for both)
            const float up = max_groups(top);
            const bool move = up > st[mt].over;
            const float d = move ? up : 0.0f;
            const Factor by(st[mt].over == kSlack ? -d : 0.0f);   // (nothing to scale at the first move)
            st[mt].m += d;
            st[mt].over = move ? kSlack : st[mt].over;
            st[mt].l = by.divisor(st[mt].l);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) st[mt].o[e] *= by.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] -= d;
            if (small != 0) {
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st[mt].l += small_share(y[4 * a + i], hs[a].lv(i), hs[a].iv(i));
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float p0 = __builtin_amdgcn_exp2f(y[4 * a + i]);
                const float p1 = __builtin_amdgcn_exp2f(y[4 * a + i + 1]);
                st[mt].l = __builtin_fmaf(p0, hs[a].iv(i), st[mt].l);
                st[mt].l = __builtin_fmaf(p1, hs[a].iv(i + 1), st[mt].l);
                const at_f32x2 pp{p0, p1};
                const at_f16x2 ph = __builtin_convertvector(pp, at_f16x2);
                p[mt][4 * a + i] = ph[0], p[mt][4 * a + i + 1] = ph[1];
            }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
        at_f16x8 vf[4];
        value_operands<D>(t, w, vf);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                st[mt].o[4 * w + e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[e], p[mt], st[mt].o[4 * w + e], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The waves' states joined through LDS, then the unit's rows written: bf16
// rows where this workgroup saw all of the unit's keys (part == NULL), else a
// part.
template <int D, int MT, int PART = kAllKeys, class Row>
__device__ __forceinline__ void finish(const AttendArgs& a, RowState<D> (&st)[MT], float* sh, float* part, Row row_of) {
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
            sm[(wave * 16 + c) * 2] = l > 0.0f ? st[mt].m : kNoRef;
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
            const Factor by(sm[(w * 16 + r) * 2] - m);
            sum += by.divisor(sm[(w * 16 + r) * 2 + 1]);
            const float* src = so + (w * 16 + r) * kStride + d0;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) o[e] = __builtin_fmaf(by.f, src[e], o[e]);
        }
        const int64_t row = row_of(mt * 16 + r);   // row * Hq + head, -1 past the unit
        if (row < 0) continue;
        if (PART == kSharedKeys && !part) {
            float* dst = a.prior + row * (D + kPriorTail);
#pragma unroll
            for (int e = 0; e < D / 16; e += 4)
                *reinterpret_cast<at_f32x4*>(dst + d0 + e) = at_f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]};
            if (d0 == 0) dst[D] = m, dst[D + 1] = sum;
        } else if (!part) {
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
#pragma unroll
            for (int e = 0; e < D / 16; e += 4)
                *reinterpret_cast<at_f32x4*>(part + (size_t)(mt * 16 + r) * D + d0 + e) = at_f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]};
            if ((threadIdx.x & 15) == 0) {
                float* ml = part + (size_t)16 * MT * D + (mt * 16 + r) * 2;
                ml[0] = m;
                ml[1] = sum;
            }
        }
    }
}

// Two waves hold the registers of a tile on its way beside one in use; 64
// dimensions and 16 rows fit three.  (Three at D = 128 and 16 rows spilled: 64
// decoding sequences of up to 16,384 tokens 264 against 218 us.)
constexpr int waves_per_simd(int D, int MT) { return MT == 1 && D == 64 ? 3 : 2; }

template <int D, int MT>
constexpr size_t finish_lds() {
    return (size_t)(kWaves * 16 * (D + 4) + kWaves * 16 * 2) * 4;
}

// Dense work is cut evenly over the workgroups whatever the sequences'
// lengths are.  Sequence b has units (key/value head, row tile): its rows
// times the G heads of a key/value head, flattened as (row, head), 16 MT a
// tile; each counts kUnitTiles for what a unit costs whatever it reads, then
// its key tiles, those its last row sees.  All units of all sequences lie on
// one line, and workgroup w takes [w per, (w + 1) per) of it, across unit
// borders.  A unit whose tiles lie in one workgroup's range is written at once;
// the parts of the others are joined by a second launch.  A workgroup leaves
// at most two parts: a later one of the unit its range begins in (slot 2 w),
// and the first one of the unit that goes on past its end (slot 2 w + 1).
//
// (Without the unit's own cost, 480 units of one tile each went eight to a
// workgroup, one after the other: 60 us.)
constexpr int kUnitTiles = 8;
constexpr int kWhole = 32;   // units of up to this cost are not cut further than the card needs
struct SeqWork {
    SeqRows sr;
    int tiles;       // key tiles per unit, at least 1 (a unit that sees nothing is one empty tile)
    int row_tiles;
    __device__ __forceinline__ int64_t cost() const { return (int64_t)kUnitTiles + tiles; }
};

// Key tiles of the rows at positions pos_lo .. pos_hi: [0, sink_tiles) and
// from win_tile0 on, tiles in all; keys below n_sink or in [lo, hi) are seen.
// (`own`: the first key that a sequence sees for itself.)
struct KeyRange32 {
    int lo, hi, sink_tiles, win_tile0, tiles;
};
template <int PART>
__device__ __forceinline__ KeyRange32 key_range(const AttendArgs& a, int pos_lo, int pos_hi, int own) {
    KeyRange32 k;
    k.hi = min(max(pos_hi + 1, 0), a.bt.max_pages << a.c.page_shift);
    k.lo = a.window > 0 ? min(max(max(pos_lo, 0) - a.window + 1, 0), k.hi) : 0;
    if constexpr (PART == kOwnKeys) k.lo = min(own, k.hi);
    k.sink_tiles = a.window > 0 ? (min(a.n_sink, k.lo) + kTile - 1) / kTile : 0;
    k.win_tile0 = max(k.lo / kTile, k.sink_tiles);
    k.tiles = k.sink_tiles + max((k.hi + kTile - 1) / kTile - k.win_tile0, 0);
    return k;
}

template <int MT, int PART>
__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int b) {
    SeqWork w;
    w.sr = batch_rows<PART>(a, b);
    const int n = w.sr.r1 - w.sr.r0, end = w.sr.pos0 + n;
    w.row_tiles = (int)(((int64_t)n * a.G + 16 * MT - 1) / (16 * MT));
    // no row tile sees more: all tiles up to the last row's, or with a window
    // the sinks' and those that the window of its rows' positions can touch
    const int64_t all = (min(max(end, 0), a.bt.max_pages << a.c.page_shift) + kTile - 1) / kTile;
    int64_t most = all;
    if (a.window > 0) {
        const int span = min(n, uniform((16 * MT + a.G - 1) / a.G) + 1);
        most = min(all, ((int64_t)a.n_sink + kTile - 1) / kTile + ((int64_t)a.window + span + kTile - 2) / kTile + 1);
    }
    if constexpr (PART == kSharedKeys) most = (shared_keys(a, b) + kTile - 1) / kTile;
    if constexpr (PART == kOwnKeys) most -= own_from(a, b) / kTile;
    w.tiles = max((int)most, 1);
    return w;
}

constexpr int kPlanSeqs = 64 * kWaves;   // sequences looked at together
struct PlanLds {
    int64_t wave[kWaves];
    int largest;   // cost of the largest unit, up to kWhole + 1
};

// Where a workgroup stands: the place reached on the line, and the sequence
// there with its own place.  It lives in LDS and is read again for every unit:
// in registers over a unit's loop it would cost that loop spills.
struct Place {
    int64_t at, first;
    int b;
};

// Work of sequence b (0 past the batch).
template <int MT, int PART>
__device__ __forceinline__ int64_t work_of(const AttendArgs& a, int b) {
    if (b >= batch_size<PART>(a)) return 0;
    const SeqWork w = seq_work<MT, PART>(a, b);
    return w.cost() * w.row_tiles * a.c.Hkv;
}

// Inclusive scan over the workgroup's threads; total of all in `sum`.
__device__ __forceinline__ int64_t block_scan(int64_t x, PlanLds& ls, int64_t& sum) {
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
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) x += ls.wave[w];
        sum += ls.wave[w];
    }
    return x;
}

template <int D, int MT>
__device__ __forceinline__ void load_queries(const AttendArgs& a, at_bf16x8 (&q)[MT][D / 32], int64_t (&row)[MT], int g) {
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
}

// ------------------------------------------------------------ dense keys

// One unit's key tiles [t0, t1) against its rows [f0, f1) (flattened).
template <int D, int MT, int PART>
__device__ __forceinline__ void dense_unit(const AttendArgs& a, const SeqRows& sr, int b, int h, int f0, int f1,
                                           const KeyRange32& kr, int t0, int t1, int own, float* sh, float* part) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int pos_lo = PART == kSharedKeys ? kr.hi - 1 : sr.pos0 + uniform(f0 / a.G);
    const int pos_hi = PART == kSharedKeys ? kr.hi - 1 : sr.pos0 + uniform((f1 - 1) / a.G);
    auto row_of = [&](int r) -> int64_t {
        const int f = f0 + r;
        if (f >= f1) return -1;
        const int i = f / a.G;
        return (int64_t)(sr.r0 + i) * a.Hq + h * a.G + (f - i * a.G);
    };
    at_bf16x8 q[MT][D / 32];
    int64_t row[MT];
    int pos[MT];
    RowState<D> st[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        row[mt] = row_of(mt * 16 + c);
        pos[mt] = row[mt] < 0 ? -1 : PART == kSharedKeys ? kr.hi - 1 : sr.pos0 + (f0 + mt * 16 + c) / a.G;
        st[mt].m = 0.0f;
        st[mt].over = -INFINITY;
        st[mt].l = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) st[mt].o[e] = at_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // the first wave of the unit's first part begins from the shared keys' sums
        if (PART == kOwnKeys && t0 == 0 && wave == 0 && row[mt] >= 0 && own > 0) {
            const float* src = a.prior + row[mt] * (D + kPriorTail);
            const float m = src[D], l = src[D + 1];   // (without a key: zeros, and no reference)
            st[mt].m = l > 0.0f ? m : 0.0f;
            st[mt].over = l > 0.0f ? kSlack : -INFINITY;
            st[mt].l = g == 0 ? l : 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < D / 16; ++e) st[mt].o[e][r] = src[(4 * g + r) * (D / 16) + e];
        }
    }
    load_queries<D, MT>(a, q, row, g);
    auto query = [&](int mt, int j) { return q[mt][j]; };

    const int32_t* table = batch_table<PART>(a, b);
    const int page = 1 << a.c.page_shift;
    // the wave's steps are the tiles t0 + wave, t0 + wave + kWaves, ..; a lane
    // holds the page of one half of one of the next 32
    PageLanes pl;
    auto key0_of = [&](int t) { return (t < kr.sink_tiles ? t : kr.win_tile0 + t - kr.sink_tiles) * kTile; };
    auto tile_of = [&](int n) { return t0 + wave + n * kWaves; };
    auto lane_key = [&](int block) {
        const int t = tile_of(32 * block + (lane >> 1));
        return t < t1 ? key0_of(t) + 16 * (lane & 1) : -1;
    };
    // (a page with no visible key is not looked at: its scale and bytes may be anything)
    auto seen = [&](int key) { return (key < kr.hi) & ((key + 15 >= kr.lo) | (key < a.n_sink)); };
    struct Where {
        int key0, pid[2];   // page of each half, -1 when it has none
    };
    auto load = [&](KvTile<D>& t, Where& w, int n) {
        if (n % 32 == 0) pl.turn(table, a, h, n / 32, lane_key, seen);
        w.key0 = key0_of(tile_of(n));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            w.pid[x] = pl.page(2 * (n % 32) + x);
            const size_t tile = (size_t)max(w.pid[x], 0) * a.c.Hkv + h;
            const size_t base = ((tile << a.c.page_shift) + ((w.key0 + 16 * x) & (page - 1))) * D;
            const uint8_t* kp = a.c.k + base;
            const uint8_t* vp = a.c.v + base;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                t.k[x][j] = *reinterpret_cast<const at_u32x4*>(kp + (c * D + 64 * j + 16 * g));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* p = vp + ((4 * g + i) * D + c * (D / 16));
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
    uint32_t small = 0;
    auto scales = [&](PageScale (&hs)[2], int n) {   // before the loads of step n + 1, which may turn the lanes
        if (n % 32 == 0) pl.scales(a.c2);
        hs[0] = pl.scale(2 * (n % 32));
        hs[1] = pl.scale(2 * (n % 32) + 1);
        small = pl.any_small(2 * (n % 32), 2);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto step = [&](KvTile<D>& t, const Where& w, const PageScale (&hs)[2]) {
        const int last = w.key0 + kTile - 1;
        bool whole;
        if constexpr (PART == kOwnKeys) {   // (no window)
            whole = w.pid[0] >= 0 && w.pid[1] >= 0 && last <= pos_lo && last < kr.hi && w.key0 >= kr.lo;
        } else {
            whole = w.pid[0] >= 0 && w.pid[1] >= 0 && last <= pos_lo && last < kr.hi &&
                    (a.window <= 0 || w.key0 > pos_hi - a.window || last < a.n_sink);
        }
        if (!whole) {
            // bytes of keys that no row sees may be NaN: their weights are 0, so the values must be finite
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = w.key0 + 16 * x + 4 * g + i;
                    const bool ok = (w.pid[x] >= 0) & (key < kr.hi) & ((key >= kr.lo) | (key < a.n_sink));
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) t.v[4 * x + i][j] = ok ? t.v[4 * x + i][j] : 0u;
                }
        }
        tile_step<D, MT>(t, query, hs, st, !whole, small, [&](int mt, int x, int i) {
            const int key = w.key0 + 16 * x + 4 * g + i;
            const int from = PART == kOwnKeys ? kr.lo - 1 : a.window > 0 ? max(pos[mt], 0) - a.window : -1;
            return (w.pid[x] >= 0) & (key <= pos[mt]) & (key < kr.hi) &
                   ((key > from) | (key < a.n_sink));
        });
    };

    const int steps = (t1 - t0 - wave + kWaves - 1) / kWaves;
    if (steps > 0) {
        KvTile<D> ta, tb;
        Where wa, wb;
        PageScale hs[2];
        pl.read(table, a, 0, lane_key);
        load(ta, wa, 0);
        for (int n = 0;; n += 2) {   // a step's keys and values are loaded during the step before
            scales(hs, n);
            if (n + 1 < steps) load(tb, wb, n + 1);
            step(ta, wa, hs);
            if (n + 1 >= steps) break;
            scales(hs, n + 1);
            if (n + 2 < steps) load(ta, wa, n + 2);
            step(tb, wb, hs);
            if (n + 2 >= steps) break;
        }
    }
    finish<D, MT, PART>(a, st, sh, part, row_of);
}

template <int D, int MT, int PART>
__global__ __launch_bounds__(64 * kWaves, (waves_per_simd(D, MT))) void attend_kernel(AttendArgs a) {
    const int n_batch = batch_size<PART>(a);
    if constexpr (PART == kSharedKeys) note_own(a);
    extern __shared__ __attribute__((aligned(16))) float sh[];
    __shared__ PlanLds ls;
    __shared__ Place place;
    // the total, then the sequence that this workgroup's range begins in; one
    // look at up to kPlanSeqs sequences serves both
    if (threadIdx.x == 0) ls.largest = 0;
    __syncthreads();
    int64_t total = 0, sum, w0 = 0, x0 = 0;
    for (int b0 = 0; b0 < n_batch; b0 += kPlanSeqs) {
        w0 = work_of<MT, PART>(a, b0 + threadIdx.x);
        x0 = total + (n_batch > 1 ? block_scan(w0, ls, sum) : (sum = work_of<MT, PART>(a, 0)));
        if (w0 > 0) atomicMax(&ls.largest, (int)min(seq_work<MT, PART>(a, b0 + threadIdx.x).cost(), (int64_t)kWhole + 1));
        total += uniform(sum);
    }
    __syncthreads();
    const int largest = uniform(ls.largest);
    // (at least 1: a batch whose sequences have no rows has no work)
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)(largest <= kWhole ? max(largest, 1) : kMinPer));
    const int64_t begin = (int64_t)blockIdx.x * per, end = min(begin + per, total);
    Crossing* crossing = reinterpret_cast<Crossing*>(a.head) + 2 * (int64_t)blockIdx.x;
    if (threadIdx.x == 0) crossing[0].n = crossing[1].n = 0;
    if (begin >= end) return;
    if (n_batch <= kPlanSeqs) {
        if (x0 - w0 <= begin && begin < x0) place = Place{begin, x0 - w0, (int)threadIdx.x};
    } else {
        int64_t before = 0;
        for (int b0 = 0; b0 < n_batch; b0 += kPlanSeqs) {
            const int64_t w = work_of<MT, PART>(a, b0 + threadIdx.x), x = before + block_scan(w, ls, sum);
            if (x - w <= begin && begin < x) place = Place{begin, x - w, b0 + (int)threadIdx.x};
            before += uniform(sum);
            if (begin < before) break;
        }
    }
    __syncthreads();
    while (true) {
        const int b = uniform(place.b);
        const int64_t at = uniform(place.at), first = uniform(place.first);
        const SeqWork w = seq_work<MT, PART>(a, b);
        const int units = w.row_tiles * a.c.Hkv, u = uniform((int)((at - first) / w.cost()));
        const int64_t us = first + u * w.cost(), tile0 = us + kUnitTiles;   // places of the unit and of its first tile
        const int64_t stop = min(end, us + w.cost());
        const int h = uniform(u / w.row_tiles), f0 = (u - h * w.row_tiles) * 16 * MT;
        const int f1 = min(f0 + 16 * MT, (w.sr.r1 - w.sr.r0) * a.G);
        const int t0 = (int)max(at - tile0, (int64_t)0), t1 = (int)max(stop - tile0, (int64_t)0);
        float* part = nullptr;
        if (t0 > 0 || t1 < w.tiles) part = a.part + ((int64_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * part_floats<D, 16 * MT>();
        if (part && t0 < t1 && threadIdx.x == 0) {
            const int w0 = (int)(tile0 / per), w1 = (int)((tile0 + w.tiles - 1) / per);
            crossing[t0 > 0 ? 0 : 1] = Crossing{w1 - w0 + 1, (int)blockIdx.x - w0, 2 * w0 + 1, w0 + 1, {w.sr.r0, f0, f1, h}};
        }
        __syncthreads();
        if (threadIdx.x == 0) {   // the next unit
            Place n{stop, first, b};
            if (u + 1 == units && stop == us + w.cost() && stop < end) {
                n.first += units * w.cost();
                do ++n.b;
                while (seq_work<MT, PART>(a, n.b).row_tiles == 0);
            }
            place = n;
        }
        if (t0 < t1) {   // (else the range ends before the unit's first tile)
            const int all = PART == kSharedKeys ? shared_keys(a, b) - 1 : 0;   // position that the shared keys end at
            const int own = PART == kOwnKeys ? own_from(a, b) : 0;
            const KeyRange32 kr = key_range<PART>(a, PART == kSharedKeys ? all : w.sr.pos0 + uniform(f0 / a.G),
                                                  PART == kSharedKeys ? all : w.sr.pos0 + uniform((f1 - 1) / a.G), own);
            dense_unit<D, MT, PART>(a, w.sr, b, h, f0, f1, kr, t0, min(t1, kr.tiles), own, sh, part);
        }
        __syncthreads();   // finish() has read its LDS
        if (uniform(place.at) >= end) return;
    }
}

// ------------------------------------------------------------ listed keys

// Entries of the staged list: rows of the cache for the unit's head, the
// constants of their pages, and (packed) the group's rows that see them.
struct ListLds {
    int32_t row[kListChunk];
    float c[kListChunk], lv[kListChunk], iv[kListChunk];
    uint32_t mask[kListChunk];
};

// (row, head) pairs of a group that share a list, and the units of 16 MT they
// make: a group is one row with a list of its own, or `group` rows of a packed
// list.
__host__ __device__ __forceinline__ int list_tiles(int group, int G, int RT) { return (group * G + RT - 1) / RT; }

// A unit is 16 MT (row, head) pairs of one group and key/value head, flattened
// as elsewhere; its list is idx[row], or with PACKED the group's entries that
// one of the unit's rows sees.
template <int D, int MT, bool PACKED>
__global__ __launch_bounds__(64 * kWaves, (waves_per_simd(D, MT))) void attend_list_kernel(AttendArgs a) {
    extern __shared__ __attribute__((aligned(16))) float sh[];
    ListLds& ls = *reinterpret_cast<ListLds*>(sh);
    __shared__ int s_cnt[kWaves];
    __shared__ int s_small;   // the staged list holds keys of small value scales
    constexpr int RT = 16 * MT;
    const int group = PACKED ? a.group : 1;
    UnitRows u;
    u.h = uniform((int)(blockIdx.x % a.c.Hkv));
    int rest = uniform((int)(blockIdx.x / a.c.Hkv));
    const int split = uniform(rest % a.splits);
    rest = uniform(rest / a.splits);
    const int ht = list_tiles(group, a.G, RT), tile = uniform(rest % ht), grp = uniform(rest / ht);
    u.r0 = grp * group;
    u.f0 = tile * RT;
    u.f1 = min(u.f0 + RT, min(group, a.T - u.r0) * a.G);
    if (u.f0 >= u.f1) return;
    int b = 0, pos0;   // position of row u.r0
    if constexpr (PACKED) {
        pos0 = max(a.bt.len[0], 0) - a.T + u.r0;
    } else {
        b = uniform(row_seq(a.bt, u.r0, a.T));
        const SeqRows sr = seq_rows(a.bt, b, a.T);
        if (u.r0 < sr.r0 || u.r0 >= sr.r1) return;
        pos0 = sr.pos0 + (u.r0 - sr.r0);
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int32_t* list = a.list + (size_t)grp * a.cap;
    const uint32_t* masks = PACKED ? a.masks + (size_t)grp * a.cap : nullptr;
    const int n = PACKED ? min(max(a.lens[grp], 0), a.cap) : a.cap;
    const int per = uniform((n + a.splits - 1) / a.splits);
    const int e0 = split * per, e1 = min(e0 + per, n);
    if (split > 0 && e0 >= e1) return;
    const int used = max((n + per - 1) / max(per, 1), 1);
    const int i0 = uniform(u.f0 / a.G), i1 = uniform((u.f1 - 1) / a.G);   // the unit's first and last row in the group
    const uint32_t rows = (~0u << i0) & (~0u >> (31 - i1));

    auto row_of = [&](int r) -> int64_t { return out_row(a, u, u.f0 + r); };
    at_bf16x8 q[MT][D / 32];
    int64_t row[MT];
    int qi[MT];   // the lane's row in the group
    RowState<D> st[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        row[mt] = row_of(mt * 16 + c);
        qi[mt] = row[mt] < 0 ? 0 : (u.f0 + mt * 16 + c) / a.G;
        st[mt].m = 0.0f;
        st[mt].over = -INFINITY;
        st[mt].l = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) st[mt].o[e] = at_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    load_queries<D, MT>(a, q, row, g);
    auto query = [&](int mt, int j) { return q[mt][j]; };
    const int32_t* table = a.bt.table + (size_t)b * a.bt.max_pages;
    const int page = 1 << a.c.page_shift;
    const int end = min(max(pos0 + i1 + 1, 0), a.bt.max_pages << a.c.page_shift);   // keys the unit's rows may see

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
    auto step = [&](KvTile<D>& x, int at, int cnt, uint32_t small) {
        KeyScale hs[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int k = at + 16 * z + 4 * g;
            hs[z].c_ = *reinterpret_cast<const at_f32x4*>(ls.c + k);
            hs[z].lv_ = *reinterpret_cast<const at_f32x4*>(ls.lv + k);
            hs[z].iv_ = *reinterpret_cast<const at_f32x4*>(ls.iv + k);
        }
        // (padded entries repeat the last key; packed, they have no rows; a unit of one row sees every other entry)
        if constexpr (PACKED) {
            const at_u32x4 m0 = *reinterpret_cast<const at_u32x4*>(ls.mask + at + 4 * g);
            const at_u32x4 m1 = *reinterpret_cast<const at_u32x4*>(ls.mask + at + 16 + 4 * g);
            tile_step<D, MT>(x, query, hs, st, i1 > i0 || at + kTile > cnt, small,
                             [&](int mt, int z, int i) { return (((z == 0 ? m0 : m1)[i] >> qi[mt]) & 1u) != 0; });
        } else {
            tile_step<D, MT>(x, query, hs, st, at + kTile > cnt, small,
                             [&](int, int z, int i) { return at + 16 * z + 4 * g + i < cnt; });
        }
    };

    for (int c0 = e0; c0 < e1; c0 += kListChunk) {
        // the chunk's keys, compacted in list order
        const int c1 = min(c0 + kListChunk, e1);
        int cnt = 0;
        __syncthreads();   // the previous chunk has been read
        if (threadIdx.x == 0) s_small = 0;
        for (int s0 = c0; s0 < c1; s0 += 64 * kWaves) {
            const int e = s0 + threadIdx.x;
            int s = -1;
            uint32_t m = rows;
            if (e < c1) {
                s = list[e];
                if constexpr (PACKED) {   // rows at or after the key only
                    const int later = s - pos0;
                    m &= masks[e];
                    if (later > 0) m &= later < 32 ? ~0u << later : 0u;
                    if (m == 0u) s = -1;
                }
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
                const size_t pg = (size_t)pid * a.c.Hkv + u.h;
                ls.row[at] = (int)((pg << a.c.page_shift) + (s & (page - 1)));
                const PageScale ps = page_scale(a.c2, a.c.ks[pg], a.c.vs[pg]);
                ls.c[at] = ps.c_, ls.lv[at] = ps.lv_, ls.iv[at] = ps.iv_;
                if (is_small(ps)) s_small = 1;
                if constexpr (PACKED) ls.mask[at] = m;
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
            ls.mask[at] = 0u;
        }
        __syncthreads();
        const uint32_t small = uniform(s_small);
        KvTile<D> ta, tb;
        int at = wave * kTile;
        constexpr int kStep = kWaves * kTile;
        if (at < cnt) {
            load(ta, at);
            while (true) {
                const bool more = at + kStep < cnt;
                if (more) load(tb, at + kStep);
                step(ta, at, cnt, small);
                if (!more) break;
                at += kStep;
                const bool more2 = at + kStep < cnt;
                if (more2) load(ta, at + kStep);
                step(tb, at, cnt, small);
                if (!more2) break;
                at += kStep;
            }
        }
    }
    __syncthreads();   // the list is done with: finish() reuses its LDS
    const int64_t slot = (((int64_t)grp * ht + tile) * a.c.Hkv + u.h) * a.splits + split;
    finish<D, MT>(a, st, sh, used > 1 ? a.part + slot * part_floats<D, 16 * MT>() : nullptr, row_of);
}

// ------------------------------------------------------- joining the splits

// One workgroup per query row and head.
template <int D, int MT, bool PACKED>
__global__ __launch_bounds__(kJoinRows * D / 4) void attend_list_join_kernel(AttendArgs a) {
    constexpr int RT = 16 * MT;
    const int64_t r = blockIdx.x;   // row * Hq + head
    const int t = (int)(r / a.Hq), head = (int)(r % a.Hq), h = head / a.G, g = head - h * a.G;
    if constexpr (!PACKED) {
        if (t < cu_at(a.bt, 0, a.T) || t >= cu_at(a.bt, a.bt.n_seq, a.T)) return;
    }
    const int group = PACKED ? a.group : 1, grp = t / group, ht = list_tiles(group, a.G, RT);
    const int n = PACKED ? min(max(a.lens[grp], 0), a.cap) : a.cap;
    const int per = (n + a.splits - 1) / a.splits, used = (n + per - 1) / max(per, 1);
    if (used <= 1) return;   // written by its only workgroup
    const int f = (t - grp * group) * a.G + g;
    const int64_t slot0 = (((int64_t)grp * ht + f / RT) * a.c.Hkv + h) * a.splits;
    join_wide<D, RT>(a, r, f % RT, used, slot0, slot0 + 1, 1);
}

template <int D, int MT, int PART>
hipError_t launch_part(const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    attend_kernel<D, MT, PART><<<(unsigned)p.blocks, 64 * kWaves, finish_lds<D, MT>(), st>>>(a);
    if (p.join) launch_join<D, 16 * MT, PART>(p, a, st);
    return hipGetLastError();
}

template <int KIND, int D, int MT>
hipError_t launch(const AttendPlan& p, const AttendArgs& a, hipStream_t st, int part) {
    const int64_t rows = (int64_t)a.T * a.Hq;
    if constexpr (KIND == LTK_ATTEND) {
        return part == kAllKeys      ? launch_part<D, MT, kAllKeys>(p, a, st)
               : part == kSharedKeys ? launch_part<D, MT, kSharedKeys>(p, a, st)
                                     : launch_part<D, MT, kOwnKeys>(p, a, st);
    } else {
        constexpr size_t lds = std::max(finish_lds<D, MT>(), sizeof(ListLds));
        constexpr bool packed = KIND == LTK_ATTEND_PACKED;
        attend_list_kernel<D, MT, packed><<<(unsigned)p.blocks, 64 * kWaves, lds, st>>>(a);
        if (p.join) attend_list_join_kernel<D, MT, packed><<<(unsigned)rows, kJoinRows * D / 4, 0, st>>>(a);
    }
    return hipGetLastError();
}

template <int KIND, int D>
hipError_t launch_rows(const AttendPlan& p, const AttendArgs& a, hipStream_t st, int part) {
    return p.mt == 1 ? launch<KIND, D, 1>(p, a, st, part) : launch<KIND, D, 2>(p, a, st, part);
}

template <int KIND>
hipError_t launch_kind(int D, const AttendPlan& p, const AttendArgs& a, hipStream_t st, int part) {
    return D == 64 ? launch_rows<KIND, 64>(p, a, st, part) : launch_rows<KIND, 128>(p, a, st, part);
}

}  // namespace

namespace {

constexpr size_t part_bytes(int D) { return (size_t)(D + 2) * 16 * sizeof(float); }   // of 16 rows

// attend_kernel with units of 16 mt rows; `units` bounds their number.
AttendPlan few_rows_plan(int mt, int64_t units, int D, int64_t entries) {
    AttendPlan p{};
    p.mt = mt;
    // One range of key tiles a workgroup, and as many workgroups as run at
    // once.  (64 heads on 8, D = 128, twice as many against that: one row
    // over 65,536 tokens 37 against 33 us, 16 rows of as many sequences of up
    // to 4,096 30 against 25, 256 rows 223 against 215; D = 64, 200 rows of 32
    // heads, sequences of up to 3,000: 1,024 workgroups 81 us, 768 69, 512 76.)
    const int64_t tiles = (entries + kTile - 1) / kTile;
    const int64_t most = (std::min(units, kManyUnits) * (tiles + kUnitTiles) + kMinPer - 1) / kMinPer;
    p.blocks = std::max<int64_t>(1, std::min<int64_t>(most, 256 * waves_per_simd(D, mt)));
    p.join = p.blocks > 1;
    p.head_bytes = crossing_bytes(p.blocks);
    p.ws_bytes = p.head_bytes + (p.join ? (size_t)p.blocks * 2 * mt * part_bytes(D) : 0);
    return p;
}

// Lists of `pairs` (row, head) pairs each: packed groups of many pairs go to the
// tile kernels, attend_list_kernel takes the others.
AttendPlan list_plan(bool packed, int64_t groups, int64_t pairs, int Hkv, int D, int64_t entries) {
    if (packed && pairs > 96) return attend_tile_list_plan(groups, pairs, Hkv, D, entries);
    AttendPlan p{};
    p.mt = pairs > 16 ? 2 : 1;
    const int64_t units = groups * ((pairs + 16 * p.mt - 1) / (16 * p.mt)) * Hkv;
    // Lists are cut only while the units leave CUs with less than two workgroups,
    // each part at least one 32-key tile a wave (580 units of 2,048 keys,
    // D = 128: 54 us whole, 68 us cut in two and joined).
    const int64_t most = std::max<int64_t>(1, (entries + kTile * kWaves - 1) / (kTile * kWaves));
    p.splits = (int)std::min<int64_t>(most, std::max<int64_t>(1, 512 / std::max<int64_t>(units, 1)));
    p.blocks = units * p.splits;
    p.join = p.splits > 1;
    p.ws_bytes = std::max<size_t>(256, p.join ? (size_t)p.blocks * p.mt * part_bytes(D) : 0);
    return p;
}

// Dense calls of fewer (row, head) pairs times keys of the table than this stay
// with attend_kernel: units of 32 rows fill the card where those of 128 do not.
// (Hq 32, Hkv 8, one sequence's first 512 tokens, 2^23: 20 against 38 us; Hq 64,
// 128 rows after 1,920 tokens, 2^24: 31 against 46; Hq 32, 512 rows after 1,536,
// 2^25: 57 against 49, eight sequences of 128 rows and 1,024 tokens, 2^25: 97
// against 48.)
constexpr int64_t kTileWork = (int64_t)1 << 24;

}  // namespace

AttendPlan attend_plan(int kind, int T, int Hq, int Hkv, int D, int n_seq, int64_t entries, int group) {
    const int G = Hq / Hkv;
    // The tile kernels from 65 rows a sequence and head, or 97 (row, head) pairs
    // a group.  (Hq 64, Hkv 8, D 128, against these kernels: one sequence of
    // 131,072 tokens, 64 rows 117 against 76 us, 96 rows 107 against 136, 512
    // rows 339 against 399; 32 sequences of 2,048 tokens, 72 rows 67 against 99,
    // 256 rows 91 against 250.  Packed, 512 rows of 1,024 keys, groups of four
    // rows, 32 pairs, 116 against 59 us, of eight 75 against 66, of 12 89 against
    // 74, of 16 97 against 85; 2,048 rows of 2,048 keys in groups of 16, 128
    // pairs, 464 against 667; at D 64, 1,024 rows in groups of 16 80 against 97.)
    if (kind == LTK_ATTEND_SELECTED) return list_plan(false, T, G, Hkv, D, entries);
    if (kind == LTK_ATTEND_PACKED)
        return list_plan(true, ((int64_t)T + group - 1) / group, (int64_t)group * G, Hkv, D, entries);
    const int64_t rows = (int64_t)T * G, seqs = std::max(n_seq, 1), work = (int64_t)T * Hq * entries;
    if (rows > 64 * seqs && work > kTileWork) {
        const int waves = attend_tile_wide(rows, n_seq, work) ? 8 : 4;
        return attend_tile_plan(waves, (rows / (32 * waves) + n_seq) * Hkv, D, entries);
    }
    // Rows that share keys: 16 or 32 to a unit.  (64 rows in one unit read
    // the cache once but leave one wave on a SIMD: eight rows of 64 heads on
    // 8 over 1,048,576 tokens took 529 us so, and 507 us as two units of 32
    // whose ranges run side by side and meet in L2; with units of 16, 760.)
    const int mt = rows > 16 * seqs ? 2 : 1;
    return few_rows_plan(mt, (rows / (16 * mt) + n_seq) * Hkv, D, entries);
}

// Calls of less work may need more: lists are cut while units are few, and the
// dense kernels' parts differ.  For lists the largest over all numbers of groups
// that are cut; for dense calls that of each kernel that a smaller call can reach,
// each of which grows with rows, sequences and entries.
size_t attend_workspace_bound(int kind, int T, int Hq, int Hkv, int D, int n_seq, int64_t entries, int group) {
    const int G = Hq / Hkv;
    size_t most = attend_plan(kind, T, Hq, Hkv, D, n_seq, entries, group).ws_bytes;
    if (kind != LTK_ATTEND) {
        const bool packed = kind == LTK_ATTEND_PACKED;
        const int64_t groups = packed ? ((int64_t)T + group - 1) / group : T;
        for (int64_t g = 1; g <= groups; ++g) {
            const AttendPlan p = list_plan(packed, g, packed ? (int64_t)group * G : G, Hkv, D, entries);
            most = std::max(most, p.ws_bytes);
            if (p.blocks / p.splits > 256) break;   // (no list is cut from here on)
        }
        return most;
    }
    const int64_t rows = (int64_t)T * G, seqs = std::max(n_seq, 1), work = (int64_t)T * Hq * entries;
    if (G <= 16 * seqs)
        most = std::max(most, few_rows_plan(1, (std::min(rows / 16, seqs) + seqs) * Hkv, D, entries).ws_bytes);
    if (rows > 16) most = std::max(most, few_rows_plan(2, (rows / 32 + seqs) * Hkv, D, entries).ws_bytes);
    if (rows > 64 && work > kTileWork)
        most = std::max(most, attend_tile_plan(4, (rows / 128 + seqs) * Hkv, D, entries).ws_bytes);
    if (attend_tile_wide(rows, 1, work)) most = std::max(most, attend_tile_plan(8, (rows / 256 + seqs) * Hkv, D, entries).ws_bytes);
    return most;
}

hipError_t launch_attend(int kind, int D, const AttendPlan& p, AttendArgs& a, void* ws, hipStream_t st, int part) {
    a.splits = p.splits;
    a.head = ws;
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.head_bytes);
    if (p.tile) return launch_attend_tile(kind, D, p, a, st, part);
    if (kind == LTK_ATTEND) return launch_kind<LTK_ATTEND>(D, p, a, st, part);
    if (kind == LTK_ATTEND_SELECTED) return launch_kind<LTK_ATTEND_SELECTED>(D, p, a, st, part);
    return launch_kind<LTK_ATTEND_PACKED>(D, p, a, st, part);
}

}  // namespace ltk
