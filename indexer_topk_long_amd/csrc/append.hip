// append.hip -- appending rows to the paged e4m3 cache on gfx950, with the
// position rotation applied on the way.
//
// Rotation of the pair (a, b) at position p and frequency f:
//   a' = a cos(p f) - b sin(p f),   b' = b cos(p f) + a sin(p f).
// The angle is formed in turns, p f / 2pi, as an unevaluated sum of two
// doubles whose whole turns are dropped before the sine: at position 2^20 the
// fp32 angle would be off by 0.06 radians.
//
// Keys are rotated in fp64 and rounded once to fp32: with an fp32 rotation
// about one key byte in a million would fall on the other side of an e4m3
// rounding border.  fp64 FMAs issue at the rate of fp32 ones here, and each
// key is rotated once.  Queries outnumber keys Hq / Hkv to one and are
// rounded to bf16, whose half step is 2^16 times fp32's: they are rotated in
// fp32 with the sine and cosine of the exactly reduced angle.
//
// One workgroup takes one page of one key/value head for keys or values (all
// rows of the call that fall into the page), so the page's largest magnitude
// is a workgroup reduction and each row is read once, kept in registers and
// written once.  The workgroups behind those rotate the queries.
//
// Bound by the bytes where rows are many: 8,192 rows of 64 query and 8
// key/value heads, D = 128 (319 MB read and written) take 77 us, 4.1 TB/s of
// the 5.0 that a large copy reaches.  Bound by the chain page id, scale, sines,
// reduction, store where they are few: one row takes 4.6 us, 96 rows of as many
// sequences 8 us.
#include <algorithm>

#include "attend.hpp"

namespace ltk {

namespace {

struct AppendArgs {
    KvCache c;
    KvBatch bt;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q;
    uint16_t* q_out;
    const double* inv_freq;
    int T, Hq, rot, interleaved;
    int units;       // pages that can receive rows, upper bound
    int heads_per;   // query heads per thread
};

// p * f in turns, reduced to [-1/2, 1/2]
__device__ __forceinline__ double turns(int p, double f) {
    constexpr double kInv2Pi = 0.15915494309189535, kInv2PiLo = -9.839338337591243e-18;
    const double r = f * kInv2Pi;
    const double re = __builtin_fma(f, kInv2Pi, -r) + f * kInv2PiLo;
    const double x = (double)p;
    const double t = x * r;
    const double te = __builtin_fma(x, r, -t) + x * re;
    const double y = (t - __builtin_rint(t)) + te;   // te passes a turn where t passes 2^52
    return y - __builtin_rint(y);
}

// Least power of two s (as its exponent) with amax <= 448 s, in [-64, 64].
__device__ __forceinline__ int scale_exp(float amax) {
    if (!(amax > 0.0f)) return -64;
    int e;
    const float m = frexpf(amax, &e);              // amax = m 2^e, m in [1/2, 1)
    const int s = (m <= 0.875f) ? e - 9 : e - 8;   // 448 = 0.875 * 2^9
    return min(max(s, -64), 64);
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    auto sat = [](float x) { return __builtin_amdgcn_fmed3f(x, -kE4m3Max, kE4m3Max); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), w, true);
}

// x c and x / s (s > 0) in fp32 rounded to odd: an inexact result whose last bit
// is 0 moves to its neighbour on the exact value's side.  Rounding that to e4m3
// gives the exact value rounded once.
__device__ __forceinline__ float to_odd(float y, float rest, bool away) {   // rest: exact value less y (its sign)
    const uint32_t b = __float_as_uint(y);
    return rest == 0.0f || (b & 1u) ? y : __uint_as_float(away ? b + 1u : b - 1u);
}
__device__ __forceinline__ float product_to_odd(float x, float c) {   // c > 0
    const float y = x * c, rest = __builtin_fmaf(x, c, -y);
    return to_odd(y, rest, (rest < 0.0f) == (x < 0.0f));
}
__device__ __forceinline__ float quotient_to_odd(float x, float s) {
    const float y = x / s, rest = __builtin_fmaf(-y, s, x);
    return to_odd(y, rest, (rest < 0.0f) == (x < 0.0f));
}

// VEC bf16 values
template <int VEC>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&x)[VEC]) {
    if constexpr (VEC == 8) {
        const at_u32x4 w = *reinterpret_cast<const at_u32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
    } else if constexpr (VEC == 4) {
        const at_u32x2 w = *reinterpret_cast<const at_u32x2*>(p);
#pragma unroll
        for (int i = 0; i < 2; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
    } else {
        x[0] = __uint_as_float((uint32_t)*p << 16);
    }
}
template <int VEC>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&x)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<at_u32x4*>(p) =
            at_u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<at_u32x2*>(p) = at_u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    } else {
        *p = (uint16_t)pack_bf16(x[0], 0.0f);
    }
}
template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&x)[VEC], float inv) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<at_u32x2*>(p) =
            at_u32x2{pack_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                     pack_e4m3(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv)};
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint32_t*>(p) = pack_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    } else {
        *p = (uint8_t)pack_e4m3(x[0] * inv, 0.0f, 0.0f, 0.0f);
    }
}

// A row is cut into items of two VEC-element vectors: item i of the rotated
// part holds VEC whole pairs (its vectors lie rot/2 apart, or side by side
// when pairs are interleaved); past rot the vectors are side by side.  VEC
// divides rot / 2, so that no vector crosses rot.
struct Item {
    int lo, hi, freq;   // element offsets; first frequency index, -1 past rot
};
template <int VEC>
__device__ __forceinline__ Item item_of(int i, int rot, int interleaved) {
    const int at = 2 * VEC * i;
    if (at >= rot) return Item{at, at + VEC, -1};
    if (interleaved) return Item{at, at + VEC, VEC * i};
    return Item{VEC * i, VEC * i + rot / 2, VEC * i};
}

// The item's pairs rotated in place; F is double (keys) or float (queries).
// cs[j] is the cosine and sine of the item's j-th frequency.
template <int VEC, typename F>
__device__ __forceinline__ void rotate_item(float (&lo)[VEC], float (&hi)[VEC], const F (&c)[VEC], const F (&s)[VEC],
                                            int interleaved) {
    auto rot = [](float& a, float& b, F cc, F ss) {
        const F x = (F)a, y = (F)b;
        if constexpr (sizeof(F) == 8) {
            a = (float)__builtin_fma(x, cc, -(y * ss));
            b = (float)__builtin_fma(y, cc, x * ss);
        } else {
            a = __builtin_fmaf(x, cc, -(y * ss));
            b = __builtin_fmaf(y, cc, x * ss);
        }
    };
    if (!interleaved) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) rot(lo[j], hi[j], c[j], s[j]);
    } else if constexpr (VEC == 1) {
        rot(lo[0], hi[0], c[0], s[0]);
    } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            rot(lo[2 * j], lo[2 * j + 1], c[j], s[j]);
            rot(hi[2 * j], hi[2 * j + 1], c[VEC / 2 + j], s[VEC / 2 + j]);
        }
    }
}

// With few rows (decode) a page's items keep 8 threads a row busy, each with
// VEC sines in turn: then all threads form the rows' sines together, through
// LDS (96 sequences of one row, 32 query heads, pages of 16: 10.1 -> 8 us; more
// rows fill the threads as they are).
constexpr int kShareRows = 4;

// One page, one key/value head, keys or values.  NT threads, NI items each:
// NT * NI >= page * D / (2 VEC).
template <int D, int VEC, int NT, int NI>
__device__ __forceinline__ void append_page(const AppendArgs& a, int unit, int h, bool is_v) {
    __shared__ float s_max[NT / 64];
    __shared__ double s_cs[kShareRows][D / 2][2];
    constexpr int kItems = D / (2 * VEC);
    const int tid = threadIdx.x, page = 1 << a.c.page_shift;
    const int b = unit_seq(a.bt, unit, a.T, 1, page, 2);
    const SeqRows sr = seq_rows(a.bt, b, a.T);
    const int end = sr.pos0 + (sr.r1 - sr.r0);               // the sequence's length
    const int nth = unit - unit_first(a.bt, b, a.T, 1, page, 2);
    const int P = (max(sr.pos0, 0) >> a.c.page_shift) + nth;
    if (sr.r1 == sr.r0 || nth < 0 || P >= a.bt.max_pages) return;
    const int p0 = max(max(sr.pos0, 0), P << a.c.page_shift);
    if (p0 >= end) return;
    const int p1 = min(end, (P + 1) << a.c.page_shift), rows = p1 - p0;
    const int pid = a.bt.table[(size_t)b * a.bt.max_pages + P];
    const uint16_t* src = is_v ? a.v : a.k;
    const int slot0 = p0 & (page - 1);
    const int rot = is_v ? 0 : a.rot;

    float lo[NI][VEC], hi[NI][VEC];
    float top = 0.0f;
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        const int w = n * NT + tid, r = w / kItems;
        const Item it = item_of<VEC>(w % kItems, rot, a.interleaved);
#pragma unroll
        for (int j = 0; j < VEC; ++j) lo[n][j] = hi[n][j] = 0.0f;
        if (r < rows) {
            const uint16_t* p = src + ((size_t)(sr.r0 + (p0 - sr.pos0) + r) * a.c.Hkv + h) * D;
            load_bf16<VEC>(p + it.lo, lo[n]);
            load_bf16<VEC>(p + it.hi, hi[n]);
        }
    }
    const bool share = rows <= kShareRows && rot > 0;
    if (share) {
        for (int i = tid; i < rows * (rot / 2); i += NT) {
            const int r = i / (rot / 2), f = i - r * (rot / 2);
            sincospi(2.0 * turns(p0 + r, a.inv_freq[f]), &s_cs[r][f][1], &s_cs[r][f][0]);
        }
        __syncthreads();
    }
    // (the page id is first needed here: rows and sines do not wait for it)
    if (pid < 0 || pid >= a.c.n_pages) return;
    const size_t tile = (size_t)pid * a.c.Hkv + h;            // the page's and head's tile
    float* scale = (is_v ? a.c.vs : a.c.ks) + tile;
    uint8_t* dst = (is_v ? a.c.v : a.c.k) + ((tile << a.c.page_shift) * D);
    const float old = slot0 > 0 ? *scale : 0.0f;
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        const int w = n * NT + tid, r = w / kItems;
        const Item it = item_of<VEC>(w % kItems, rot, a.interleaved);
        if (r < rows && it.freq >= 0) {
            double c[VEC], s[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (share)
                    c[j] = s_cs[r][it.freq + j][0], s[j] = s_cs[r][it.freq + j][1];
                else
                    sincospi(2.0 * turns(p0 + r, a.inv_freq[it.freq + j]), &s[j], &c[j]);
            }
            rotate_item<VEC, double>(lo[n], hi[n], c, s, a.interleaved);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) top = fmaxf(top, fmaxf(fabsf(lo[n][j]), fabsf(hi[n][j])));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((tid & 63) == 0) s_max[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) top = fmaxf(top, s_max[w]);

    const float need = ldexpf(1.0f, scale_exp(top));
    const float now = fmaxf(need, old);
    if (tid == 0 && now != old) *scale = now;
    if (slot0 > 0 && now > old) {   // the page's earlier tokens move to the grown scale
        const float f = old / now;   // exact: a scale that grows is a power of two
        for (int i = tid; i < slot0 * (D / 16); i += NT) {
            at_u32x4 w = reinterpret_cast<const at_u32x4*>(dst)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const auto x = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
                const auto y = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
                w[j] = pack_e4m3(product_to_odd(x[0], f), product_to_odd(x[1], f), product_to_odd(y[0], f),
                                 product_to_odd(y[1], f));
            }
            reinterpret_cast<at_u32x4*>(dst)[i] = w;
        }
    }
    // scales written here are powers of two; a page begun by another writer may keep another one
    const bool pow2 = (__float_as_uint(now) & 0x7fffffu) == 0u;
    if (!pow2) {
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int j = 0; j < VEC; ++j) lo[n][j] = quotient_to_odd(lo[n][j], now), hi[n][j] = quotient_to_odd(hi[n][j], now);
    }
    const float inv = pow2 ? 1.0f / now : 1.0f;
#pragma unroll
    for (int n = 0; n < NI; ++n) {
        const int w = n * NT + tid, r = w / kItems;
        const Item it = item_of<VEC>(w % kItems, rot, a.interleaved);
        if (r >= rows) continue;
        uint8_t* p = dst + (size_t)(slot0 + r) * D;
        store_e4m3<VEC>(p + it.lo, lo[n], inv);
        store_e4m3<VEC>(p + it.hi, hi[n], inv);
    }
}

// Queries: thread = (row, block of heads, item), items fastest.
template <int D, int VEC, int NT>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, int blk) {
    constexpr int kItems = D / (2 * VEC);
    const int hb = (a.Hq + a.heads_per - 1) / a.heads_per;
    const int64_t w = (int64_t)blk * NT + threadIdx.x;
    const int i = (int)(w % kItems), h0 = (int)(w / kItems % hb) * a.heads_per;
    const int64_t row64 = w / kItems / hb;
    if (row64 >= a.T) return;
    const int row = (int)row64;
    const SeqRows sr = seq_rows(a.bt, row_seq(a.bt, row, a.T), a.T);
    if (row < sr.r0 || row >= sr.r1) return;
    const int pos = sr.pos0 + (row - sr.r0);
    const Item it = item_of<VEC>(i, a.rot, a.interleaved);
    float c[VEC], s[VEC];
    if (it.freq >= 0) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) sincospif((float)(2.0 * turns(pos, a.inv_freq[it.freq + j])), &s[j], &c[j]);
    }
    const int h1 = min(h0 + a.heads_per, a.Hq);
    for (int h = h0; h < h1; ++h) {
        const size_t at = ((size_t)row * a.Hq + h) * D;
        float x[VEC], y[VEC];
        load_bf16<VEC>(a.q + at + it.lo, x);
        load_bf16<VEC>(a.q + at + it.hi, y);
        if (it.freq >= 0) rotate_item<VEC, float>(x, y, c, s, a.interleaved);
        store_bf16<VEC>(a.q_out + at + it.lo, x);
        store_bf16<VEC>(a.q_out + at + it.hi, y);
    }
}

template <int D, int VEC, int NT, int NI>
__global__ __launch_bounds__(NT) void kv_append_kernel(AppendArgs a) {
    const int kv_blocks = a.units * a.c.Hkv * 2;
    const int blk = blockIdx.x;
    if (blk < kv_blocks) {
        const int h = blk % a.c.Hkv, rest = blk / a.c.Hkv;
        append_page<D, VEC, NT, NI>(a, rest >> 1, h, rest & 1);
    } else {
        rotate_queries<D, VEC, NT>(a, blk - kv_blocks);
    }
}

// Threads of a workgroup for items of VEC elements.
constexpr int append_threads(int D, int vec, int page) {
    const int items = page * D / (2 * vec), most = vec == 1 ? 1024 : 256;   // single elements: more threads, not more registers
    return items < 64 ? 64 : (items > most ? most : items);
}

template <int D, int VEC, int PAGE>
hipError_t launch_page(const AppendArgs& a, unsigned blocks, hipStream_t st) {
    constexpr int NT = append_threads(D, VEC, PAGE);
    constexpr int NI = (PAGE * D / (2 * VEC) + NT - 1) / NT;
    kv_append_kernel<D, VEC, NT, NI><<<blocks, NT, 0, st>>>(a);
    return hipGetLastError();
}

template <int D, int VEC>
hipError_t launch_vec(const AppendArgs& a, unsigned blocks, hipStream_t st) {
    switch (a.c.page_shift) {
        case 4: return launch_page<D, VEC, 16>(a, blocks, st);
        case 5: return launch_page<D, VEC, 32>(a, blocks, st);
        case 6: return launch_page<D, VEC, 64>(a, blocks, st);
        default: return launch_page<D, VEC, 128>(a, blocks, st);
    }
}

}  // namespace

AppendPlan append_plan(int T, int Hq, int Hkv, int D, int n_seq, int page, int rot, bool queries) {
    AppendPlan p{};
    // rot / 2 (half-split pairs) and rot (the border) in whole vectors
    p.vec = rot % 16 == 0 ? 8 : rot % 8 == 0 ? 4 : 1;
    // a thread's sines serve up to 8 heads while the threads left still fill the
    // card (8,192 rows of 64 heads, D = 128: 107 us with 1, 83 with 2, 76 with 4,
    // 74 with 8, 80 with 16; 96 rows of 32 heads: 10.0 us with 1, 12.3 with 8)
    p.heads_per = 1;
    while (p.heads_per < 8 && (int64_t)T * Hq * (D / 16) / (2 * p.heads_per) >= 1 << 18) p.heads_per *= 2;
    const int nt = append_threads(D, p.vec, page);
    const int64_t units = unit_bound(n_seq, T, 1, page, 2), hb = (Hq + p.heads_per - 1) / p.heads_per;
    if (units > 0x7fffffff) return p;   // (fits: false)
    p.units = (int)units;
    p.blocks = units * Hkv * 2 + (queries ? ((int64_t)T * hb * (D / (2 * p.vec)) + nt - 1) / nt : 0);
    p.fits = grid_fits(p.blocks, nt);
    return p;
}

hipError_t launch_kv_append(const AppendPlan& p, const KvCache& c, const KvBatch& bt, int D, const uint16_t* k,
                            const uint16_t* v, const uint16_t* q, int T, int Hq, const double* inv_freq, int rot,
                            int interleaved, uint16_t* q_out, hipStream_t st) {
    AppendArgs a{};
    a.c = c;
    a.bt = bt;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.inv_freq = inv_freq;
    a.T = T;
    a.Hq = Hq;
    a.rot = rot;
    a.interleaved = interleaved;
    a.units = p.units;
    a.heads_per = p.heads_per;
    const unsigned blocks = (unsigned)p.blocks;
    if (p.vec == 8) return D == 64 ? launch_vec<64, 8>(a, blocks, st) : launch_vec<128, 8>(a, blocks, st);
    if (p.vec == 4) return D == 64 ? launch_vec<64, 4>(a, blocks, st) : launch_vec<128, 4>(a, blocks, st);
    return D == 64 ? launch_vec<64, 1>(a, blocks, st) : launch_vec<128, 1>(a, blocks, st);
}

}  // namespace ltk
