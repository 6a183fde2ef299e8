// attend_tile.hip -- attention over the paged e4m3 cache for many rows per key
// on gfx950 (prefill chunks, packed groups): bound by the matrix cores and the
// exponentials beside them.
//
// A workgroup of four or eight waves takes 128 or 256 (row, head) pairs of one
// key/value head, 32 a wave, and 64 keys a step.  The formulas are those of
// attend.hip; what differs is where the conversions happen.  Each key byte meets
// all the workgroup's rows, so keys and values are converted once per workgroup
// on their way into LDS (keys to bf16, values to fp16, both exact) and not in
// every wave:
//  - keys [64][D] bf16, read as rows of v_mfma_f32_32x32x16_bf16;
//  - values transposed, [D][64] fp16: a thread loads 4 bytes of 8 keys, pairs
//    them byte by byte and stores four 16-byte pieces, so the second product
//    reads its operand with one ds_read_b128.  The 8 keys are those whose
//    weights one lane holds after the first product, so weights go from the
//    first product's result to the second's operand in place.
// Two stages of LDS (64 KB at D = 128) and one barrier a step; the bytes of the
// step after next are on their way in registers, and with eight waves or at
// D = 64 those of the step behind it too, though not without a pause: there every
// second step forms the constants of the pages at its head (PageLanes::scales,
// whose branch the compiler turns into selects) and with them waits for every
// load in flight.  Two waves run on a SIMD: two workgroups of four waves
// or one of eight on a CU.
//
// Three chunks of up to 1,999 tokens after up to 16,384 (32 heads on 8, D = 128,
// 7.9e11 operations) take 850 to 910 us, 870 to 930 TFLOP/s of the 1,200 that a
// large matrix product reaches, at the 1.85 GHz that the card holds under that
// load: the matrix units are busy 42 % of the cycles, and 30 % of the waves'
// cycles are waits, the one above among them.
// 2,048 rows with a window of 4,096 (32 heads on 4, D = 64) take 116 to 131 us,
// 530 to 590 TFLOP/s: half the products for the same exponentials.  Packed, 128
// groups of 16 rows of 2,048 keys each (64 heads on 8, D = 128) take 442 to 484
// us: every key of a group's list, 2.3 times a row's own, goes through the
// products of all its rows, and each wave reads every key's constants and masks
// beside its operands (2.4 LDS instructions a matrix instruction, 1.1 above).
#include <algorithm>
#include <atomic>

#include "attend_join.hpp"

namespace ltk {

namespace {

typedef float at_f32x16 __attribute__((ext_vector_type(16)));
typedef int at_i32x4 __attribute__((ext_vector_type(4)));

constexpr int kKeys = 64;       // keys of a step
// A workgroup of NW waves takes 32 NW (row, head) pairs.
template <int NW>
constexpr int kRows = 32 * NW;
constexpr int kListWaves = 4;   // packed lists: 128 pairs a unit
constexpr int kRing = 256;      // list entries resolved together (one a thread), two such chunks in LDS
constexpr int kMinKeys = 4 * kKeys;   // least keys of a workgroup's range
constexpr int kUnitKeys = 4 * kKeys;  // what a unit costs whatever it reads
constexpr int kWhole = 16 * kKeys;    // units of up to this cost are not cut further than the card needs
// Units have 256 rows, of eight waves, from this many rows a sequence and this
// many (row, head) pairs times keys of the table, else 128.  (Hq 64, Hkv 8,
// D 128, units of 128 against 256: one sequence of 131,072 tokens, 128 rows a
// head 111 against 158 us, 256 rows 194 against 174, 1,024 rows 640 against
// 596; 32 sequences of 2,048 tokens, 128 rows 68 against 83, 256 rows 115
// against 91.  Hq 32, one sequence with 512 rows: 2,048 tokens 51 against 54 us,
// 8,192 107 against 105.)
constexpr int kWide = 256;
constexpr int64_t kWideWork = (int64_t)1 << 25;

__device__ __forceinline__ float max_halves(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// A stage of LDS: keys [64][D] bf16, then values [D][64] fp16.  16-byte chunk
// x of a row lies at chunk x ^ swizzle(row), so that the 16 lanes of one LDS
// cycle (256 bytes) touch all banks: 16 consecutive rows when read, 2 or 4 key
// rows and 16 value rows 4 apart when written.  A 256-byte row (keys at
// D = 128) takes its number; of 128-byte rows two fill the banks, and pairs
// take theirs.  Rows are whole numbers of 128 bytes, so within a row a chunk
// is exchanged by one XOR on the byte offset.
template <int D>
constexpr int kStageBytes = 4 * kKeys * D;
template <int D>
constexpr int kValuesAt = 2 * kKeys * D;
struct Ring {                     // listed keys, resolved
    int32_t row[2 * kRing];       // cache row of the unit's head, -1: no key
    uint32_t mask[2 * kRing];     // rows that see it
    float c[2 * kRing], lv[2 * kRing], iv[2 * kRing];
    int small[2 * kRing / kKeys];   // of a step's keys, some have small value scales
};
__device__ __forceinline__ uint8_t* lds() {
    extern __shared__ at_u32x4 lds_words[];
    return reinterpret_cast<uint8_t*>(lds_words);
}
template <int D>
__device__ __forceinline__ int key_swizzle(int key) {
    return D == 128 ? key & 15 : (key >> 1) & 7;
}
__device__ __forceinline__ int val_swizzle(int d) { return ((d >> 1) & 7) ^ ((d >> 4) & 1); }
// An offset that the compiler does not see through: what is derived from it is
// formed again in every step, by an XOR each, and not kept in registers over
// the loop.
__device__ __forceinline__ int per_step(int off) {
    asm volatile("" : "+v"(off));
    return off;
}

// The thread's part of a step's bytes: two 16-byte key pieces, one value patch
// (8 keys x 4 bytes), or both.  256 threads can hold the patches of D = 128 and
// half as many pieces: four waves take both there.  At D = 64, and with eight
// waves, the first waves take the values and the next the keys.  Waves w and
// w + 4 share a SIMD, so at D = 128 with eight waves every SIMD has the same
// work; at D = 64 two waves take the values and two the keys, and of eight the
// other four neither.
template <int D, int NW>
struct Part {
    static constexpr int kPatches = 2 * D;            // threads that take a value patch, and as many key pieces
    static constexpr bool kBoth = 64 * NW < 2 * kPatches;
    static constexpr int kPieces = D / 16;            // 16-byte pieces of a key row
    bool keys, vals;
    int key, piece;          // key pieces: rows key and key + 32
    int chunk, dq;           // value patch: 8 keys of chunk, dimensions 4 dq ..
    __device__ __forceinline__ Part() {
        const int tid = threadIdx.x;
        vals = kBoth || tid < kPatches;
        keys = kBoth || (tid >= kPatches && tid < 2 * kPatches);
        const int i = tid & (kPatches - 1);
        key = i / kPieces, piece = i % kPieces;
        chunk = i / (D / 4), dq = i % (D / 4);
    }
    // the patch's i-th key: its chunk holds the keys of one lane's weights
    __device__ __forceinline__ int val_key(int i) const {
        return 16 * (chunk >> 1) + 4 * (chunk & 1) + (i & 3) + ((i & 4) << 1);
    }
};
// Where a thread takes either, both share the same registers.
template <bool BOTH>
struct Raw {
    at_u32x4 w[BOTH ? 4 : 2];
    __device__ __forceinline__ at_u32x4& k(int i) { return w[i]; }
    __device__ __forceinline__ uint32_t v(int i) const { return w[(BOTH ? 2 : 0) + i / 4][i % 4]; }
    __device__ __forceinline__ void set_v(int i, uint32_t x) { w[(BOTH ? 2 : 0) + i / 4][i % 4] = x; }
};

// The conversions of a step's bytes into the stage at LDS offset `stage`, in
// four equal parts (i = 0 .. 3) that the matrix instructions of the step
// before are issued between.
template <int D, int NW>
__device__ __forceinline__ void store_stage(const Part<D, NW>& p, Raw<Part<D, NW>::kBoth>& r, int stage, int i) {
    if (i < 2) {
        if (!p.keys) return;
        // rows key and key + 32, chunks 2 piece and 2 piece + 1
        const int at = per_step(p.key * (2 * D) + (((2 * p.piece) ^ key_swizzle<D>(p.key)) << 4)) + stage;
        *reinterpret_cast<at_bf16x8*>(lds() + at + i * (64 * D)) = bf16_of(r.k(i)[0], r.k(i)[1]);
        *reinterpret_cast<at_bf16x8*>(lds() + (at ^ 16) + i * (64 * D)) = bf16_of(r.k(i)[2], r.k(i)[3]);
        return;
    }
    if (!p.vals) return;
    const int e = 2 * (i - 2);   // bytes e and e + 1 of the patch: value rows 4 dq + e and the next
    at_f16x8 o0, o1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = __builtin_amdgcn_perm(r.v(2 * j + 1), r.v(2 * j), e ? 0x07030602u : 0x05010400u);
        const at_f16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
        const at_f16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
        o0[2 * j] = x0[0], o0[2 * j + 1] = x0[1];
        o1[2 * j] = x1[0], o1[2 * j + 1] = x1[1];
    }
    const int at = per_step(p.dq * 512 + ((p.chunk ^ val_swizzle(4 * p.dq)) << 4)) + stage + kValuesAt<D>;
    const int pair = at ^ ((e >> 1) << 4);   // both rows' chunk
    *reinterpret_cast<at_f16x8*>(lds() + pair + e * 128) = o0;
    *reinterpret_cast<at_f16x8*>(lds() + pair + (e + 1) * 128) = o1;
}

// Running state of a wave's 32 rows: lane (c, g) = (lane % 32, lane / 32)
// holds row c, of its accumulators the dimensions 32 t + 8 (r / 4) + 4 g + r % 4.
template <int D>
struct WaveState {
    float m, over, l;
    at_f32x16 o[D / 32];
};

// 64 keys of a stage against the wave's rows, in two halves of 32.
//
// A wave issues in order, and a matrix instruction keeps its unit busy for 8
// issue slots: the vector work of one half is written between the matrix
// instructions of the other, and the next stage's conversions between those
// of the last product (about 8 vector instructions each).  The scheduling
// barriers hold that order; left alone, the compiler puts each product in one
// run, and both waves of a SIMD then wait for the same unit in turn.
//   scores 0 | scores 1 with weights of 0 | values 0 with weights of 1 | values 1 with fill
// LDS operands are read kAhead instructions before their use.
//
// scale(hb, i, m, c, lv): constants of the lane's keys 4 i .. 4 i + 3 of half
// hb (i < 4), lv less m; scale.inverse: their 1 / vs; scale.small(hb), not 0:
// some of the half's value scales may be small (the same in all lanes).  mask.each(hb, i, y)
// hides keys among four, mask.late(hb, x) among all 16 where it says so.
constexpr int kAhead = 4;
template <int D, class Scale, class Mask, class Fill>
__device__ __forceinline__ void step_keys(int stage, const at_bf16x8 (&q)[D / 16], WaveState<D>& st, Scale scale,
                                          Mask mask, Fill fill) {
    const int lane = threadIdx.x & 63, c = lane & 31, g = lane >> 5;
    constexpr int N = D / 16;   // matrix instructions of a product of one half
    at_f32x16 x0, x1;
    at_f16x8 p[4];
    // operand n of the 4 N: keys n = N hb + j, then values n = 2 N + N hb + (D / 32) w + t
    at_u32x4 frag[kAhead];
    const int k0 = per_step(c * (2 * D) + ((g ^ key_swizzle<D>(c)) << 4)) + stage;
    const int v0 = per_step(c * 128 + ((g ^ val_swizzle(c)) << 4)) + stage + kValuesAt<D>;
    auto fetch = [&](int n) {
        if (n >= 4 * N) return;
        const int w = (n - 2 * N) / (D / 32), t = (n - 2 * N) % (D / 32);
        // key row 32 hb + c, chunk 2 j + g; value row 32 t + c, chunk 2 w + g
        const int at = n < 2 * N ? (k0 ^ (32 * (n % N))) + 64 * D * (n / N) : (v0 ^ (32 * w)) + 4096 * t;
        frag[n % kAhead] = *reinterpret_cast<const at_u32x4*>(lds() + at);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i);
#pragma unroll
    for (int r = 0; r < 16; ++r) x0[r] = x1[r] = 0.0f;
    auto score = [&](int n) {
        at_f32x16& x = n < N ? x0 : x1;
        x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(at_bf16x8, frag[n % kAhead]), q[n % N], x, 0, 0, 0);
        fetch(n + kAhead);
    };
    auto value = [&](int n) {
        const int w = n / (D / 32), t = n % (D / 32);
        st.o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(at_f16x8, frag[n % kAhead]), p[w], st.o[t], 0, 0, 0);
        fetch(2 * N + n + kAhead);
    };
    float top = -INFINITY;
    auto relative = [&](int hb, at_f32x16& x, int i) {   // scores of four keys relative to the reference
        at_f32x4 cc, lv;
        scale(hb, i, st.m, cc, lv);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[4 * i + r] = __builtin_fmaf(x[4 * i + r], cc[r], lv[r]);
        mask.each(hb, i, x);
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, x[4 * i + r]);
    };
    auto settle = [&](int hb, at_f32x16& x) {   // moves the reference where a score passes it by too much
        if (mask.late(hb, x)) {
            top = -INFINITY;
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, x[r]);
        }
        const uint32_t small = scale.small(hb);
        if ((__ballot(top > st.over) | small) != 0) {   // (one branch for both)
            const float up = max_halves(top);
            const bool move = up > st.over;
            const float d = move ? up : 0.0f;
            const Factor by(st.over == kSlack ? -d : 0.0f);   // (nothing to scale at the first move)
            st.m += d;
            st.over = move ? kSlack : st.over;
            st.l = by.divisor(st.l);
#pragma unroll
            for (int t = 0; t < D / 32; ++t) st.o[t] *= by.f;
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] -= d;
            if (hb == 1) {   // half 0's weights whose product is still to come: by the fp32 factor, rounded to fp16 again
#pragma unroll
                for (int r = 0; r < 8; ++r) p[1][r] = (_Float16)((float)p[1][r] * by.f);
            }
            if (small != 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    at_f32x4 cc, lv, iv;
                    scale(hb, i, 0.0f, cc, lv);
                    scale.inverse(hb, i, iv);
#pragma unroll
                    for (int r = 0; r < 4; ++r) st.l += small_share(x[4 * i + r], lv[r], iv[r]);
                }
            }
        }
        top = -INFINITY;
    };
    auto weights = [&](int hb, const at_f32x16& x, int i) {   // of four keys
        at_f32x4 iv;
        scale.inverse(hb, i, iv);
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
            const float a = __builtin_amdgcn_exp2f(x[4 * i + r]), b = __builtin_amdgcn_exp2f(x[4 * i + r + 1]);
            st.l = __builtin_fmaf(a, iv[r], st.l);
            st.l = __builtin_fmaf(b, iv[r + 1], st.l);
            const at_f32x2 ab{a, b};
            const at_f16x2 h = __builtin_convertvector(ab, at_f16x2);
            p[2 * hb + (i >> 1)][4 * (i & 1) + r] = h[0];
            p[2 * hb + (i >> 1)][4 * (i & 1) + r + 1] = h[1];
        }
    };
#pragma unroll
    for (int n = 0; n < N; ++n) {
        score(n);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = 0; n < N / 2; ++n) {
        score(N + n);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) relative(0, x0, n * (8 / N) + i);
        __builtin_amdgcn_sched_barrier(0);
    }
    settle(0, x0);
#pragma unroll
    for (int n = 0; n < N / 2; ++n) {
        score(N + N / 2 + n);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) weights(0, x0, n * (8 / N) + i);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = 0; n < N / 2; ++n) {
        value(n);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) relative(1, x1, n * (8 / N) + i);
        __builtin_amdgcn_sched_barrier(0);
    }
    settle(1, x1);
#pragma unroll
    for (int n = 0; n < N / 2; ++n) {
        value(N / 2 + n);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) weights(1, x1, n * (8 / N) + i);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        value(N + n);
        if (n % (N / 4) == 0) fill(n / (N / 4));
        __builtin_amdgcn_sched_barrier(0);
    }
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
// NULL), else as a part.
template <int D, int NW>
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
        part[(size_t)kRows<NW> * D + 2 * r] = l > 0.0f ? st.m : kNoRef;
        part[(size_t)kRows<NW> * D + 2 * r + 1] = l;
    }
}

// ------------------------------------------------------------ dense keys

// Work is cut evenly as in attend.hip, here on a line of keys: the unit of row
// tile i counts kUnitKeys for itself and then A + i Q keys, at least as many as
// its last row sees, so that a sequence's prefix sums have a closed form.
struct SeqLine {
    SeqRows sr;
    int tiles;       // row tiles
    int64_t A, Q;
    __device__ __forceinline__ int64_t keys(int i) const { return A + i * Q; }
    __device__ __forceinline__ int64_t cost(int i) const { return kUnitKeys + keys(i); }
    __device__ __forceinline__ int64_t before(int i) const { return i * (kUnitKeys + A) + Q * ((int64_t)i * (i - 1) / 2); }
};
template <int NW>
__device__ __forceinline__ SeqLine seq_line(const AttendArgs& a, int b) {
    SeqLine s;
    s.sr = seq_rows(a.bt, b, a.T);
    const int n = s.sr.r1 - s.sr.r0;
    s.tiles = (int)(((int64_t)n * a.G + kRows<NW> - 1) / kRows<NW>);
    s.Q = uniform((kRows<NW> + a.G - 1) / a.G);
    const int64_t cap = (int64_t)a.bt.max_pages << a.c.page_shift;
    s.A = max(min((int64_t)s.sr.pos0 + 1 + s.Q, cap), (int64_t)1);
    // a window's rows see at most the sinks, the window and the tiles' borders
    const int64_t win = (int64_t)a.n_sink + a.window + s.Q + 1 + 3 * kKeys;
    if (a.window > 0 && 2 * win < 2 * s.A + s.Q * (s.tiles - 1)) s.A = win, s.Q = 0;   // where that is less in all
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

// Constants of a step's four pages, in scalar registers.  (Named, not an
// array: an indexed array ends up in scratch memory, and the wait for it is a
// wait for every load in flight.)
struct StepScales {
    PageScale s0, s1, s2, s3;
    uint32_t small;   // bit i: the value scale of page i is small
    __device__ __forceinline__ PageScale get(int i) const { return i == 0 ? s0 : i == 1 ? s1 : i == 2 ? s2 : s3; }
};
struct DenseScale {
    const StepScales& s;
    __device__ __forceinline__ void operator()(int hb, int i, float m, at_f32x4& c, at_f32x4& lv) const {
        const PageScale x = s.get(2 * hb + (i >> 1));
        const float y = x.lv_ - m;
        c = at_f32x4{x.c_, x.c_, x.c_, x.c_};
        lv = at_f32x4{y, y, y, y};
    }
    __device__ __forceinline__ void inverse(int hb, int i, at_f32x4& iv) const {
        const float x = s.get(2 * hb + (i >> 1)).iv_;
        iv = at_f32x4{x, x, x, x};
    }
    __device__ __forceinline__ uint32_t small(int hb) const { return s.small >> (2 * hb) & 3u; }
};

template <int D, int NW>
__device__ __forceinline__ void dense_unit(const AttendArgs& a, const SeqRows& sr, int b, const UnitRows& u,
                                           const KeyTiles& kt, int t0, int t1, float* part) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, g = lane >> 5;
    const int fw = u.f0 + 32 * wave;                      // the wave's rows [fw, fw1)
    const int fw1 = min(fw + 32, u.f1);
    const int pos_lo = sr.pos0 + uniform(fw / a.G), pos_hi = sr.pos0 + uniform((max(fw1, 1) - 1) / a.G);
    const int64_t row = out_row(a, u, fw + c);
    const int pos = row < 0 ? -1 : sr.pos0 + (fw + c) / a.G;
    const int from = a.window > 0 ? max(max(pos, 0) - a.window, -1) : -1;   // the lane's row sees keys behind it, and the sinks
    at_bf16x8 q[D / 16];
    WaveState<D> st;
    begin_rows<D>(a, row, q, st);

    const int32_t* table = a.bt.table + (size_t)b * a.bt.max_pages;
    const int page = 1 << a.c.page_shift;
    const Part<D, NW> p;
    auto key0_of = [&](int t) { return (t < kt.sink_tiles ? t : kt.win_tile0 + t - kt.sink_tiles) * kKeys; };
    // a lane holds the page of one 16-key group of the next 16 steps
    PageLanes pl;
    auto lane_key = [&](int block) {
        const int t = t0 + 16 * block + (lane >> 2);
        return t < t1 ? key0_of(t) + 16 * (lane & 3) : -1;
    };
    // (a page with no visible key is not looked at: its scale and bytes may be anything)
    auto seen = [&](int key) { return (key < kt.hi) & ((key + 15 >= kt.lo) | (key < a.n_sink)); };
    // What later needs to know of a step's four pages: bit i is set when keys
    // 16 i .. of the step have a page and are looked at.
    using Bytes = Raw<Part<D, NW>::kBoth>;
    auto load = [&](int t, Bytes& raw) -> int {
        const int n = t - t0, key0 = key0_of(t), at = 4 * (n % 16);
        if (n % 16 == 0) pl.turn(table, a, u.h, n / 16, lane_key, seen);
        const int p0 = pl.page(at), p1 = pl.page(at + 1), p2 = pl.page(at + 2), p3 = pl.page(at + 3);
        auto page_of = [&](int grp) { return grp == 0 ? p0 : grp == 1 ? p1 : grp == 2 ? p2 : p3; };
        // byte offset in the cache of key 16 grp of the step: scalar
        auto base = [&](int grp) -> size_t {
            return ((((size_t)max(page_of(grp), 0) * a.c.Hkv + u.h) << a.c.page_shift) + ((key0 + 16 * grp) & (page - 1))) * D;
        };
        if (p.keys) {   // a wave's pieces lie in one group, and in the second one on
            const int grp = D == 128 ? (wave & 3) >> 1 : wave & 1;
            const int off = (p.key & 15) * D + 16 * p.piece;
            raw.k(0) = *reinterpret_cast<const at_u32x4*>(a.c.k + base(grp) + off);
            raw.k(1) = *reinterpret_cast<const at_u32x4*>(a.c.k + base(grp + 2) + off);
        }
        if (p.vals) {   // D = 128: a wave's patches lie in one group; D = 64: in one a half wave
            const int off = (p.val_key(0) & 15) * D + 4 * p.dq;
            const uint8_t* v = D == 128 ? a.c.v + base(wave & 3) + off
                                        : a.c.v + (lane < 32 ? base(2 * (wave & 1)) : base(2 * (wave & 1) + 1)) + off;
#pragma unroll
            for (int i = 0; i < 8; ++i) raw.set_v(i, *reinterpret_cast<const uint32_t*>(v + (p.val_key(i) - p.val_key(0)) * D));
        }
        return (p0 >= 0 ? 1 : 0) | (p1 >= 0 ? 2 : 0) | (p2 >= 0 ? 4 : 0) | (p3 >= 0 ? 8 : 0);
    };
    auto seen_by_all = [&](int key0, int ok, int lo, int hi) {   // every key of the step by rows at lo .. hi
        return ok == 15 && key0 + kKeys - 1 <= lo && key0 + kKeys <= kt.hi &&
               (a.window <= 0 || key0 > hi - a.window || key0 + kKeys <= a.n_sink);
    };
    // what a step's bytes need before they are converted
    auto settle_raw = [&](int t, int pages, Bytes& raw) {
        if (!p.vals) return;
        const int key0 = key0_of(t);
        if (pages == 15 && key0 + kKeys <= kt.hi && (key0 >= kt.lo || key0 + kKeys <= a.n_sink)) return;
        // bytes of keys that no row sees may be NaN: their weights are 0, so the values must be finite
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int key = key0 + p.val_key(i);
            const bool ok = ((pages >> (p.chunk >> 1)) & 1) & (key < kt.hi) & ((key >= kt.lo) | (key < a.n_sink));
            raw.set_v(i, ok ? raw.v(i) : 0u);
        }
    };
    struct Mask {
        int pages;
        bool none;                  // no key of the step is hidden
        int key, last, from, n_sink;   // the lane's first key; its row sees keys up to last, behind from or below n_sink
        __device__ __forceinline__ void each(int, int, at_f32x16&) const {}
        __device__ __forceinline__ bool late(int hb, at_f32x16& y) const {
            if (none) return false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // by signs, not by 16 compares at once: their results would fill the scalar registers
                const int end = (pages >> (2 * hb + (i >> 1))) & 1 ? last : -1;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int k = key + 32 * hb + 8 * i + r;
                    const uint32_t hide = (uint32_t)(min(end - k, max(k - from - 1, n_sink - 1 - k)) >> 31);
                    y[4 * i + r] = __uint_as_float((~hide & __float_as_uint(y[4 * i + r])) | (hide & 0xff800000u));
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            return true;
        }
    };
    auto step = [&](int t, int pages, int stage, auto fill) {
        const int n = t - t0, key0 = key0_of(t), at = 4 * (n % 16);
        if (n % 16 == 0) pl.scales(a.c2);
        // (a wave none of whose rows sees the step goes through it too: a way
        // around would give its accumulators two places, and cost 70 spills)
        const StepScales sc{pl.scale(at), pl.scale(at + 1), pl.scale(at + 2), pl.scale(at + 3), pl.any_small(at, 4)};
        step_keys<D>(stage, q, st, DenseScale{sc},
                     Mask{pages, seen_by_all(key0, pages, pos_lo, pos_hi), key0 + 4 * g, min(pos, kt.hi - 1), from, a.n_sink}, fill);
    };

    // step t computes from one stage while t + 1 is written to the other and
    // the loads of t + 2 are on their way; where a thread's bytes take 8
    // registers, those of t + 3 too (but see the pause above: even steps wait
    // for all of them)
    if (t0 < t1) {
        constexpr bool kDeep = !Part<D, NW>::kBoth;
        Bytes ra, rb;
        pl.read(table, a, 0, lane_key);
        int now = load(t0, ra), next = 0, after = 0;
        settle_raw(t0, now, ra);
#pragma unroll
        for (int i = 0; i < 4; ++i) store_stage<D, NW>(p, ra, 0, i);
        if (t0 + 1 < t1) next = load(t0 + 1, ra);
        if (kDeep && t0 + 2 < t1) after = load(t0 + 2, rb);
        __syncthreads();
        auto body = [&](int t, int x, Bytes& raw) {   // raw: the bytes of t + 1
            // (past the last step the conversions write a stage that nothing reads)
            if (t + 1 < t1) settle_raw(t + 1, next, raw);
            step(t, now, x * kStageBytes<D>, [&](int i) { store_stage<D, NW>(p, raw, (x ^ 1) * kStageBytes<D>, i); });
            now = next;
            if (kDeep) {
                next = after;
                if (t + 3 < t1) after = load(t + 3, raw);
            } else if (t + 2 < t1) {
                next = load(t + 2, raw);
            }
            __syncthreads();
        };
        if constexpr (kDeep) {
            for (int t = t0;; t += 2) {
                body(t, 0, ra);
                if (t + 1 >= t1) break;
                body(t + 1, 1, rb);
                if (t + 2 >= t1) break;
            }
        } else {
            for (int t = t0; t < t1; ++t) body(t, (t - t0) & 1, ra);
        }
    }
    end_rows<D, NW>(a, row, st, part);
}

template <int NW>
struct ScanLds {
    int64_t wave[NW];
    int largest;   // cost of the largest unit, up to kWhole + 1
};
// Where a workgroup stands on the line.  It lives in LDS and is read again for
// every unit: in registers over a unit's loop it would cost that loop spills.
struct Place {
    int64_t at, first;   // on the line: the place reached, and where sequence b begins
    int b, h, i;         // sequence, head, row tile
};
template <int NW>
__device__ __forceinline__ int64_t scan_block(int64_t x, ScanLds<NW>& ls, int64_t& sum) {
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
    for (int w = 0; w < NW; ++w) {
        if (w < wave) x += ls.wave[w];
        sum += ls.wave[w];
    }
    return x;
}
template <int NW>
__device__ __forceinline__ int64_t line_of(const AttendArgs& a, int b) {
    if (b >= a.bt.n_seq) return 0;
    const SeqLine s = seq_line<NW>(a, b);
    return s.before(s.tiles) * a.c.Hkv;
}

template <int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attend_tile_kernel(AttendArgs a) {
    __shared__ ScanLds<NW> sc;
    if (threadIdx.x == 0) sc.largest = 0;
    __syncthreads();
    int64_t total = 0, sum, w0 = 0, x0 = 0;   // one look at up to 64 NW sequences gives the total and the place
    for (int b0 = 0; b0 < a.bt.n_seq; b0 += 64 * NW) {
        w0 = line_of<NW>(a, b0 + threadIdx.x);
        x0 = total + (a.bt.n_seq > 1 ? scan_block<NW>(w0, sc, sum) : (sum = line_of<NW>(a, 0)));
        if (w0 > 0) {
            const SeqLine s = seq_line<NW>(a, b0 + threadIdx.x);
            atomicMax(&sc.largest, (int)min(s.cost(s.tiles - 1), (int64_t)kWhole + 1));
        }
        total += uniform(sum);
    }
    __syncthreads();
    const int largest = uniform(sc.largest);
    // (at least 1: a batch whose sequences have no rows has no work)
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)(largest <= kWhole ? max(largest, 1) : kMinKeys));
    // Workgroups go to the eight XCDs in turn: each XCD takes a stretch of the
    // n8 ranges that hold work (so that the row tiles of one head read its keys
    // through one L2); the numbers behind those are the other workgroups'.
    const int n8 = (int)((total + 8 * per - 1) / (8 * per));
    const int me = (int)blockIdx.x < 8 * n8 ? (blockIdx.x % 8) * n8 + blockIdx.x / 8 : (int)blockIdx.x;
    const int64_t begin = me * per, end = min(begin + per, total);
    Crossing* crossing = reinterpret_cast<Crossing*>(a.head) + 2 * (int64_t)me;
    if (threadIdx.x == 0) crossing[0].n = crossing[1].n = 0;
    if (begin >= end) return;
    __shared__ Place place;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.bt.n_seq; b0 += 64 * NW) {
        if (a.bt.n_seq > 64 * NW) {
            w0 = line_of<NW>(a, b0 + threadIdx.x);
            x0 = before + scan_block<NW>(w0, sc, sum);
            before += uniform(sum);
        }
        if (x0 - w0 <= begin && begin < x0) {   // the sequence that the range begins in
            const SeqLine s = seq_line<NW>(a, b0 + threadIdx.x);
            const int64_t off = begin - (x0 - w0), head = s.before(s.tiles);
            const int h = (int)(off / head);
            int lo = 0, hi = s.tiles - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s.before(mid) <= off - h * head)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            place = Place{begin, x0 - w0, b0 + (int)threadIdx.x, h, lo};
        }
        if (begin < before) break;
    }
    __syncthreads();
    while (true) {
        const int b = uniform(place.b), h = uniform(place.h), i = uniform(place.i);
        const int64_t at = uniform(place.at);
        const SeqLine s = seq_line<NW>(a, b);
        const int64_t us = uniform(place.first) + h * s.before(s.tiles) + s.before(i);
        const int64_t key0 = us + kUnitKeys, keys = s.keys(i), stop = min(end, us + s.cost(i));
        UnitRows u;
        u.r0 = s.sr.r0;
        u.h = h;
        u.f0 = i * kRows<NW>;
        u.f1 = min(u.f0 + kRows<NW>, (s.sr.r1 - s.sr.r0) * a.G);
        // a step belongs to the range that its first key lies in
        const int64_t k0 = max(at - key0, (int64_t)0), k1 = max(stop - key0, (int64_t)0);
        float* part = nullptr;
        if (k0 > 0 || k1 < keys) part = a.part + (2 * (int64_t)me + (k0 == 0 ? 1 : 0)) * part_floats<D, kRows<NW>>();
        if (part && k0 < k1 && threadIdx.x == 0) {
            const int w0 = (int)(key0 / per), w1 = (int)((key0 + keys - 1) / per);
            crossing[k0 > 0 ? 0 : 1] = Crossing{w1 - w0 + 1, me - w0, 2 * w0 + 1, w0 + 1, u};
        }
        __syncthreads();
        if (threadIdx.x == 0) {   // the next unit
            Place n{stop, place.first, b, h, i};
            if (stop == us + s.cost(i)) {
                if (++n.i == s.tiles) n.i = 0, ++n.h;
                if (n.h == a.c.Hkv) {
                    n.h = 0;
                    n.first += a.c.Hkv * s.before(s.tiles);
                    n.b = n.at < end ? n.b + 1 : n.b;
                    while (n.at < end && seq_line<NW>(a, n.b).tiles == 0) ++n.b;
                }
            }
            place = n;
        }
        if (k0 < k1) {   // (else the range ends before the unit's first key)
            const KeyTiles kt = key_tiles(a, s.sr.pos0 + uniform(u.f0 / a.G), s.sr.pos0 + uniform((u.f1 - 1) / a.G));
            dense_unit<D, NW>(a, s.sr, b, u, kt, (int)((k0 + kKeys - 1) / kKeys),
                              min((int)((k1 + kKeys - 1) / kKeys), kt.tiles), part);
        }
        __syncthreads();
        if (uniform(place.at) >= end) return;
    }
}

// ------------------------------------------------------------ packed lists

struct ListScale {
    const Ring* r;
    int at, g, some;   // the step's place in the ring, the lane's half, the step's ring.small
    __device__ __forceinline__ int key(int hb, int i) const { return at + 32 * hb + 8 * i + 4 * g; }
    __device__ __forceinline__ void operator()(int hb, int i, float m, at_f32x4& c, at_f32x4& lv) const {
        c = *reinterpret_cast<const at_f32x4*>(r->c + key(hb, i));
        lv = *reinterpret_cast<const at_f32x4*>(r->lv + key(hb, i));
        lv = at_f32x4{lv[0] - m, lv[1] - m, lv[2] - m, lv[3] - m};
    }
    __device__ __forceinline__ void inverse(int hb, int i, at_f32x4& iv) const {
        iv = *reinterpret_cast<const at_f32x4*>(r->iv + key(hb, i));
    }
    __device__ __forceinline__ uint32_t small(int) const { return uniform(some); }
};

// A unit is 128 (row, head) pairs of one group and key/value head; its keys
// are the group's list, cut into a.splits.
template <int D>
__global__ __launch_bounds__(64 * kListWaves, 2) void attend_tile_list_kernel(AttendArgs a) {
    constexpr int NW = kListWaves;
    Ring& ring = *reinterpret_cast<Ring*>(lds() + 2 * kStageBytes<D>);
    const int ht = (a.group * a.G + kRows<NW> - 1) / kRows<NW>;   // row tiles of a group
    UnitRows u;
    u.h = uniform((int)(blockIdx.x % a.c.Hkv));
    int rest = uniform((int)(blockIdx.x / a.c.Hkv));
    const int tile = uniform(rest % ht);
    rest = uniform(rest / ht);
    const int split = uniform(rest % a.splits), grp = uniform(rest / a.splits);
    u.r0 = grp * a.group;
    u.f0 = tile * kRows<NW>;
    u.f1 = min(u.f0 + kRows<NW>, min(a.group, a.T - u.r0) * a.G);
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
    };
    auto entry_scale = [&]() {
        if (en.pid >= a.c.n_pages) en.pid = -1;
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
        const bool small = __any(is_small(ps));   // (a wave resolves the 64 entries of one step)
        if (lane == 0) ring.small[at / kKeys] = small;
    };
    const Part<D, NW> p;
    Raw<Part<D, NW>::kBoth> raw;
    uint32_t none = 0;   // bit i: the patch's i-th key is no key
    auto load = [&](int t) {
        const int at = (t * kKeys) & (2 * kRing - 1);
        if (p.keys) {
#pragma unroll
            for (int y = 0; y < 2; ++y)
                raw.k(y) = *reinterpret_cast<const at_u32x4*>(a.c.k + (size_t)max(ring.row[at + p.key + 32 * y], 0) * D +
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
                raw.set_v(i, *reinterpret_cast<const uint32_t*>(a.c.v + (size_t)max(r, 0) * D + 4 * p.dq));
            }
        }
    };
    auto settle_raw = [&]() {
        if (__any(none != 0)) {   // bytes behind no key may be NaN
#pragma unroll
            for (int i = 0; i < 8; ++i) raw.set_v(i, (none >> i) & 1u ? 0u : raw.v(i));
        }
    };
    struct Mask {
        const Ring& ring;
        int at, g, qi;
        __device__ __forceinline__ void each(int hb, int i, at_f32x16& y) const {
            const at_i32x4 m = *reinterpret_cast<const at_i32x4*>(ring.mask + at + 32 * hb + 8 * i + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // the row's bit over the whole word selects the score or -infinity
                const uint32_t see = (uint32_t)__builtin_amdgcn_sbfe(m[r], qi, 1);
                y[4 * i + r] = __uint_as_float((see & __float_as_uint(y[4 * i + r])) | (~see & 0xff800000u));
            }
        }
        __device__ __forceinline__ bool late(int, at_f32x16&) const { return false; }
    };
    auto step = [&](int t, int stage, auto fill) {
        const int at = (t * kKeys) & (2 * kRing - 1);
        step_keys<D>(stage, q, st, ListScale{&ring, at, g, ring.small[at / kKeys]}, Mask{ring, at, g, qi}, fill);
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
        settle_raw();
#pragma unroll
        for (int i = 0; i < 4; ++i) store_stage<D, NW>(p, raw, 0, i);
        if (steps > 1) load(1);
        __syncthreads();
        // a chunk's entries are read in the last two steps of the chunk two
        // before it, and resolved in the first two of the one before it
        for (int t = 0; t < steps; ++t) {
            const int x = t & 1, ph = t % kPer, chunk = t / kPer;
            if (ph == 0) entry_page();
            if (t + 1 < steps) settle_raw();
            step(t, x * kStageBytes<D>, [&](int i) { store_stage<D, NW>(p, raw, (x ^ 1) * kStageBytes<D>, i); });
            if (ph == 0) entry_scale();
            if (t + 2 < steps) load(t + 2);
            if (ph == 1) entry_store(chunk + 1);
            if (ph == 2) entry_load(chunk + 2);
            __syncthreads();
        }
    }
    const int64_t slot = (((int64_t)grp * ht + tile) * a.c.Hkv + u.h) * a.splits + split;
    end_rows<D, NW>(a, row, st, used > 1 ? a.part + slot * part_floats<D, kRows<NW>>() : nullptr);
}

// ------------------------------------------------------- joining the parts

template <int D>
__global__ __launch_bounds__(kJoinRows * D / 4) void attend_tile_list_join_kernel(AttendArgs a) {
    constexpr int NW = kListWaves;
    const int64_t r = blockIdx.x;   // row * Hq + head
    const int t = (int)(r / a.Hq), head = (int)(r % a.Hq), h = head / a.G;
    const int grp = t / a.group, ht = (a.group * a.G + kRows<NW> - 1) / kRows<NW>;
    const int n = min(max(a.lens[grp], 0), a.cap);
    const int per = ((n + kKeys - 1) / kKeys + a.splits - 1) / a.splits * kKeys;
    const int used = per > 0 ? (n + per - 1) / per : 1;
    if (used <= 1) return;
    const int f = (t % a.group) * a.G + (head - h * a.G);
    const int64_t slot0 = (((int64_t)grp * ht + f / kRows<NW>) * a.c.Hkv + h) * a.splits;
    join_wide<D, kRows<NW>>(a, r, f % kRows<NW>, used, slot0, slot0 + 1, 1);
}

template <int D, int NW>
hipError_t launch_dense(const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    attend_tile_kernel<D, NW><<<(unsigned)p.blocks, 64 * NW, 2 * kStageBytes<D>, st>>>(a);
    if (p.join) launch_join<D, kRows<NW>>(p, a, st);
    return hipGetLastError();
}

template <int D>
hipError_t launch_list(const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    constexpr size_t bytes = 2 * kStageBytes<D> + sizeof(Ring);
    if constexpr (bytes > 65536) {   // asked for once per device
        static std::atomic<uint64_t> allowed;
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        if (e != hipSuccess) return e;
        const uint64_t bit = 1ull << (dev & 63);
        if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) & bit)) {
            e = hipFuncSetAttribute(reinterpret_cast<const void*>(attend_tile_list_kernel<D>),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
            if (e != hipSuccess) return e;
            allowed.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    attend_tile_list_kernel<D><<<(unsigned)p.blocks, 64 * kListWaves, bytes, st>>>(a);
    if (p.join)
        attend_tile_list_join_kernel<D><<<(unsigned)((int64_t)a.T * a.Hq), kJoinRows * D / 4, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

bool attend_tile_wide(int64_t rows, int n_seq, int64_t work) {
    return rows >= kWide * (int64_t)std::max(n_seq, 1) && work >= kWideWork;
}

AttendPlan attend_tile_plan(int waves, int64_t units, int D, int64_t entries) {
    AttendPlan p{};
    p.tile = true;
    p.waves = waves;
    const int64_t most = (std::min(units, kManyUnits) * (entries + kKeys + kUnitKeys) + kMinKeys - 1) / kMinKeys;
    // eight waves a CU; whole rounds of the XCDs
    p.blocks = (std::max<int64_t>(1, std::min<int64_t>(most, 2048 / waves)) + 7) / 8 * 8;
    p.join = true;
    p.head_bytes = crossing_bytes(p.blocks);
    p.ws_bytes = p.head_bytes + (size_t)p.blocks * 2 * 32 * waves * (D + 2) * sizeof(float);
    return p;
}

AttendPlan attend_tile_list_plan(int64_t groups, int64_t pairs, int Hkv, int D, int64_t entries) {
    AttendPlan p{};
    p.tile = true;
    p.waves = kListWaves;
    constexpr int rows = kRows<kListWaves>;
    const int64_t units = groups * ((pairs + rows - 1) / rows) * Hkv;
    const int64_t most = (entries + kKeys - 1) / kKeys;
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(most, 512 / std::max<int64_t>(units, 1)));
    p.blocks = units * p.splits;
    p.join = p.splits > 1;
    p.ws_bytes = std::max<size_t>(256, p.join ? (size_t)p.blocks * rows * (D + 2) * sizeof(float) : 0);
    return p;
}

hipError_t launch_attend_tile(int kind, int D, const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    if (kind != LTK_ATTEND) return D == 64 ? launch_list<64>(p, a, st) : launch_list<128>(p, a, st);
    if (p.waves == 8) return D == 64 ? launch_dense<64, 8>(p, a, st) : launch_dense<128, 8>(p, a, st);
    return D == 64 ? launch_dense<64, 4>(p, a, st) : launch_dense<128, 4>(p, a, st);
}

}  // namespace ltk
