// prompt.hpp -- what the kernels over packed 16-bit prompts share: element
// types, the batch as kernels see it, its cut into units, and the tiles in LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attend.hpp"
#include "kernels_common.hpp"
#include "litetopk_prompt.h"

namespace ltk {

constexpr int kWaves = 4;    // of a workgroup
constexpr int kUnit = 32 * kWaves;   // pairs of a row tile, or keys of a key tile
constexpr int kKeys = 64;    // keys of a step (forward, dq)
constexpr int kPairs = 32;   // (row, head) pairs of a step (dk, dv)

typedef float pr_f32x16 __attribute__((ext_vector_type(16)));
typedef short pr_i16x4 __attribute__((ext_vector_type(4)));
typedef short pr_i16x8 __attribute__((ext_vector_type(8)));

// Element types: rounding of two fp32, and the matrix product of 32 rows, 32
// columns and 16 summands.  (Lane (c, g) = (lane % 32, lane / 32) holds the
// summands 8 g .. 8 g + 7 of row or column c; of the result column c, rows
// 8 (r / 4) + 4 g + r % 4.)
//
// kUp, kDown = 2^-kUp: the weights of dv's product, at most 1, are held 2^kUp times
// their size, and dv is scaled back in fp32.  fp16's normal range ends at 2^-14:
// unscaled, weights below 2^-25 (a key that no row looks at much, in a long
// sequence) would leave nothing in dv, whatever the loss is scaled by.
//
// kLift: the forward pass' weights are at most 2^kLift when its reference moves, and
// at most 2^(kLift + kSlack) until it moves again: below fp16's 65504, and as far
// above its smallest values as that allows (many small weights may be all there is
// of a result).
struct PrBf16 {
    static constexpr float kUp = 0.0f, kDown = 1.0f, kLift = 0.0f;
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16(a, b); }
    static __device__ __forceinline__ pr_f32x16 mfma(at_u32x4 a, at_u32x4 b, pr_f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(at_bf16x8, a), __builtin_bit_cast(at_bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
};
struct PrF16 {
    static constexpr float kUp = 14.0f, kDown = 0x1p-14f, kLift = 7.0f;
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const at_f32x2 x{a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, at_f16x2));
    }
    static __device__ __forceinline__ pr_f32x16 mfma(at_u32x4 a, at_u32x4 b, pr_f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(at_f16x8, a), __builtin_bit_cast(at_f16x8, b), c,
                                                      0, 0, 0);
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(at_f16x2, w)[0]; }
    static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(at_f16x2, w)[1]; }
};

struct PrRows {
    const uint16_t* p;
    int64_t row, head;   // strides in elements
};

struct PromptArgs {
    PrRows q, k, v, dout;
    const uint16_t *out_in, *rest_in;   // backward: the forward call's out and rest
    uint16_t *out, *rest, *dq, *dk, *dv;
    float* lse;
    float *lse2, *delta;      // backward, for dk and dv: [T, Hq], log2(e) lse - kUp and kDown dout . (out + rest)
    const int32_t *cu, *cu_k;
    int n_seq, T, S, Hq, Hkv, G;
    uint32_t div_g, one_g;    // ceil(2^32 / G), or 0 and all ones for G == 1
    float scale, c2;          // c2 = scale log2(e)
    int window;
    int splits, per;          // units are cut into parts of about `per` steps, `splits` of them at most
    int64_t units;            // of a key/value head
    float* part;
};

// A unit's parts: `used` of them, of `size` steps each, the last one what is left.
// (Whole ones first and the rests after them make an even load; equal parts of
// every unit: 256 units over 512 places 1.5 times the even time, these 1.3.)
struct PrParts {
    int size, used;
};
__device__ __forceinline__ PrParts pr_parts(const PromptArgs& a, int steps) {
    if (a.splits <= 1 || steps <= a.per) return PrParts{max(steps, 1), 1};
    const int n = (int)((uint32_t)(steps + a.per - 1) / (uint32_t)a.per);
    if (n <= a.splits) return PrParts{a.per, n};
    const int size = (int)((uint32_t)(steps + a.splits - 1) / (uint32_t)a.splits);
    return PrParts{size, (int)((uint32_t)(steps + size - 1) / (uint32_t)size)};
}
// The unit, part and head of a workgroup.  Heads go round the XCDs, so that a
// head's keys (dk, dv: rows) pass through one L2; first parts come before
// second ones, so that the longest come first.
struct PrPlace {
    int64_t unit;
    int part, h;
};
__device__ __forceinline__ PrPlace pr_place(const PromptArgs& a) {
    const uint32_t b = blockIdx.x, rest = b / (uint32_t)a.Hkv, part = a.splits > 1 ? rest / (uint32_t)a.units : 0u;
    return PrPlace{(int64_t)(rest - part * (uint32_t)a.units), (int)part, (int)(b - rest * (uint32_t)a.Hkv)};
}

// Quotient by G of x < G + 2^15 (exact while x (G - 1) < 2^32: G < 2^15).
__device__ __forceinline__ int pr_div_g(const PromptArgs& a, int x) {
    return (int)(__umulhi((uint32_t)x, a.div_g) + ((uint32_t)x & a.one_g));
}

// The (row, head) pairs of a key/value head are numbered f = row * G + head of
// the group.  A place among them, split once per tile; rows behind it follow by
// a small quotient.
struct PrPair {
    int i, g;
};
__device__ __forceinline__ PrPair pr_pair(const PromptArgs& a, const PrPair& base, int off) {
    const int x = base.g + off, i = pr_div_g(a, x);
    return PrPair{base.i + i, x - i * a.G};
}

// Rows and keys of a stretch of the batch: [r0, r0 + n) and [k0, k0 + m), within
// the tensors whatever cu holds.  Stretch 0 is what lies before the first
// sequence, b + 1 is sequence b, n_seq + 1 what lies behind the last one: those
// two have rows and keys that see nothing, so they are written as zeros.
struct PrSeq {
    int r0, n, k0, m;
    bool in;   // a sequence
    __device__ __forceinline__ int pos0() const { return m - n; }
};
__device__ __forceinline__ int pr_bound(const int32_t* cu, int e, int n_seq, int T) {
    return e <= 0 ? 0 : e > n_seq + 1 ? T : min(max(cu[e - 1], 0), T);
}

// Units of PER rows of a stretch (each row counting mul), without a prefix sum:
// stretch e has the numbers from  bound(e) mul / PER + e  on, at least as many as
// it can need; numbers past its own are empty.
//
// The stretch of unit u and the unit's number in it, by all lanes of a wave: 64
// stretches, or stretches of stretches, at a look, whose bounds serve for the
// result (bisection would be a chain of dependent loads).
template <int PER, bool KEYS>
__device__ __forceinline__ PrSeq pr_seq_of(const PromptArgs& a, int64_t u, int mul, int64_t& number) {
    const int lane = threadIdx.x & 63, all = a.n_seq + 2;
    auto first = [&](int bound, int e) { return (int64_t)bound * mul / PER + e; };
    auto rows = [&](int e) { return pr_bound(a.cu, e, a.n_seq, a.T); };
    auto keys = [&](int e) { return pr_bound(a.cu_k, e, a.n_seq, a.S); };
    int lo = 0, step = 1;
    while (step < (all + 63) / 64) step *= 64;
    for (; step > 1; step /= 64) {
        const int e = lo + lane * step;
        const uint64_t at = __ballot(e < all && first(KEYS ? keys(e) : rows(e), e) <= u);
        lo += at ? (63 - __clzll((long long)at)) * step : 0;
    }
    const int mine = min(lo + lane, all), r = rows(mine), k = keys(mine);
    const uint64_t at = __ballot(lo + lane < all && first(KEYS ? k : r, mine) <= u);
    const int i = at ? 63 - __clzll((long long)at) : 0, e = lo + i;
    auto bound = [&](int x, int j, bool key) {   // of stretch lo + j
        return j < 64 ? __builtin_amdgcn_readlane(x, j) : uniform(key ? keys(lo + j) : rows(lo + j));
    };
    PrSeq s;
    s.r0 = bound(r, i, false);
    s.n = max(bound(r, i + 1, false) - s.r0, 0);
    s.k0 = bound(k, i, true);
    s.m = max(bound(k, i + 1, true) - s.k0, 0);
    s.in = e >= 1 && e <= a.n_seq;
    number = u - first(KEYS ? s.k0 : s.r0, e);
    return s;
}
inline int64_t pr_units(int64_t T, int64_t mul, int per, int n_seq) { return T * mul / per + n_seq + 2; }

// A row tile: kUnit pairs of a sequence and key/value head, and the steps of
// keys that they see.
struct PrRowUnit {
    PrSeq s;
    PrPair first;   // its first pair
    int count;      // of its pairs
    int lo, hi;     // first and last position of its rows
    int t0, t1;     // steps of kKeys keys
};
__device__ __forceinline__ bool pr_row_unit(const PromptArgs& a, int64_t un, PrRowUnit& u) {
    int64_t number;
    u.s = pr_seq_of<kUnit, false>(a, un, a.G, number);
    const uint32_t pairs = (uint32_t)u.s.n * (uint32_t)a.G;   // < 2^31
    const int64_t tile = (int64_t)((pairs + kUnit - 1) / kUnit) - 1 - number;   // the longest first
    if (tile < 0) return false;
    const uint32_t f0 = (uint32_t)tile * kUnit, i = f0 / (uint32_t)a.G;
    u.first = PrPair{(int)i, (int)(f0 - i * (uint32_t)a.G)};
    u.count = (int)min(pairs - f0, (uint32_t)kUnit);
    u.lo = u.s.pos0() + u.first.i;
    u.hi = u.s.pos0() + pr_pair(a, u.first, u.count - 1).i;
    const int end = u.s.in ? min(max(u.hi + 1, 0), u.s.m) : 0;
    const int from = a.window > 0 ? min(max(max(u.lo, 0) - a.window + 1, 0), end) : 0;
    u.t0 = from / kKeys;
    u.t1 = (end + kKeys - 1) / kKeys;
    return true;
}

// A tile in LDS: rows of D 16-bit values, whose 16-byte chunk x lies at chunk
// x ^ swizzle(row), so that both ways of reading touch all banks: 16
// consecutive rows at one chunk (operands along the row), and four consecutive
// rows at four chunks (operands across rows, through the transposing read).
// A 256-byte row (D = 128) fills the banks; of 128-byte rows two do.
template <int D>
__device__ __forceinline__ int pr_swizzle(int row) {
    return D == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
}
// Operands are read at a lane's place in a tile (an offset from the start of
// LDS) with one XOR or a constant added.  The place goes through per_step in
// every step: left to itself, the compiler keeps all XORs in registers over the
// loop.
__device__ __forceinline__ int pr_per_step(int off) {
    asm volatile("" : "+v"(off));
    return off;
}
// Operands along rows: elements 16 j + 8 g .. of row 32 b + c.
template <int D>
__device__ __forceinline__ int pr_along() {
    const int lane = threadIdx.x & 63, c = lane & 31, g = lane >> 5;
    return c * (2 * D) + ((g ^ pr_swizzle<D>(c)) << 4);
}
template <int D>
__device__ __forceinline__ at_u32x4 pr_read(const uint8_t* lds, int along, int b, int j) {
    return *reinterpret_cast<const at_u32x4*>(lds + (along ^ (32 * j)) + 32 * b * (2 * D));
}
// Operands across rows: element 32 t + c of the rows 16 w + 4 g + (0 .. 3) and
// 16 w + 8 + 4 g + (0 .. 3), the rows whose scores lane (c, g) holds in
// registers 8 (w % 2) .. 8 (w % 2) + 7 of a product over 32 rows.  The
// transposing read takes four rows of 16 elements from 16 lanes (lane i: row
// i / 4, elements 4 (i % 4) ..) and gives lane i element i of the four.
template <int D>
__device__ __forceinline__ int pr_across() {
    const int lane = threadIdx.x & 63, i = lane & 15, half = (lane >> 4) & 1, g = lane >> 5;
    const int row = 4 * g + (i >> 2), chunk = 2 * half + ((i & 3) >> 1);
    return row * (2 * D) + ((chunk ^ pr_swizzle<D>(row)) << 4) + (i & 1) * 8;
}
template <int D>
__device__ __forceinline__ at_u32x4 pr_read_across(uint8_t* lds, int across, int w, int t) {
    typedef __attribute__((address_space(3))) pr_i16x4* LdsPtr;
    const int at = across ^ (64 * t);   // (the second four rows' swizzle differs in one bit)
    const pr_i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(lds + at + 16 * w * (2 * D)));
    const pr_i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(lds + (at ^ 32) + (16 * w + 8) * (2 * D)));
    const pr_i16x8 z{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    return __builtin_bit_cast(at_u32x4, z);
}
// Stores 16 elements of a row from the lanes c and c + 32 that share it: lane
// (c, g) holds 4 g .. 4 g + 3 of the first eight in (a0, a1), of the other eight
// in (b0, b1), packed.  The halves exchange words, so that each lane stores eight
// side by side.
__device__ __forceinline__ void pr_store16(uint16_t* dst, int g, uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
    const auto x = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
    *reinterpret_cast<at_u32x4*>(dst + 8 * g) = at_u32x4{x[0], y[0], x[1], y[1]};
}
// A lane's part of a row of D accumulators times f: dimensions 32 t + 8 i + 4 g ..
// in registers 4 i .. of set t.
template <class E, int D>
__device__ __forceinline__ void pr_store_row(uint16_t* dst, int g, const pr_f32x16 (&o)[D / 32], float f) {
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 8)
            pr_store16(dst + 32 * t + 2 * i, g, E::pack(o[t][i] * f, o[t][i + 1] * f), E::pack(o[t][i + 2] * f, o[t][i + 3] * f),
                       E::pack(o[t][i + 4] * f, o[t][i + 5] * f), E::pack(o[t][i + 6] * f, o[t][i + 7] * f));
}
// What rounding x and y to E's type leaves out, rounded itself.
template <class E>
__device__ __forceinline__ uint32_t pr_rest(float x, float y) {
    const uint32_t w = E::pack(x, y);
    return E::pack(x - E::lo(w), y - E::hi(w));
}
// Copies rows key0 .. key0 + 63 of one head into a tile, the last row again
// for those past the end.
template <int D>
__device__ __forceinline__ void pr_copy_tile(const PrRows& x, int64_t row0, int h, int key0, int m, uint8_t* tile) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kRowsPer = 512 / D;              // rows of a wave's copy (1 KB)
    constexpr int kCopies = 64 / kRowsPer / kWaves;  // copies of a wave
    const uint16_t* base = x.p + (row0 + key0) * x.row + (int64_t)h * x.head;
    const int last = m - 1 - key0;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int r0 = (wave * kCopies + i) * kRowsPer, r = r0 + lane / (D / 8);
        const int chunk = (lane % (D / 8)) ^ pr_swizzle<D>(r);
        const uint32_t off = (uint32_t)min(r, last) * (uint32_t)x.row * 2u + (uint32_t)chunk * 16u;
        lds_direct16_async(base, off, tile + r0 * (2 * D));
    }
}
// Waits for the direct copies into LDS that the wave has issued.
__device__ __forceinline__ void pr_wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// .. but for the newest N.
template <int N>
__device__ __forceinline__ void pr_wait_copies_but() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ float pr_max_halves(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pr_sum_halves(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

struct PromptCut {
    int64_t units, blocks;   // of a key/value head; workgroups
    int splits, per;
};
struct PromptPlan {
    PromptCut rows, grad, keys;     // the launches over row tiles (forward; dq) and over key tiles (dk, dv)
    size_t fwd_bytes, bwd_bytes;    // workspaces
    size_t stat_bytes;              // of the backward pass's: lse2, and as much for delta, before the parts
    bool fits;
};
PromptPlan prompt_plan(int T, int S, int Hq, int Hkv, int D, int n_seq, int window);
hipError_t launch_prompt(const PromptPlan& p, int type, int D, PromptArgs& a, void* ws, hipStream_t st);
hipError_t launch_prompt_backward(const PromptPlan& p, int type, int D, PromptArgs& a, void* ws, hipStream_t st);

}  // namespace ltk
