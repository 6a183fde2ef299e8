// prompt_bwd.hip -- gradients of causal attention over packed 16-bit prompts on
// gfx950: bound by the matrix cores and the vector work beside them.
//
// With P = 2^(y - lse2), lse2 = log2(e) lse, and delta = dout . (out + rest):
//   dv = P^T dout,  dP = dout v^T,  dS = P (dP - delta),
//   dq = scale dS k,  dk = scale dS^T q,
// the last two and dv summed over the query heads of a key/value head.  P and dS
// are rounded once to 16 bits for their products (operands of one type; in fp16
// dv's weights 2^14 times their size, see kUp: a step of 8,192 rows takes 2,600 us
// with and without); sums are fp32.  Two launches, so that no sum needs atomics and
// the same call gives the same bits; scores and dout v^T are formed in both, seven
// products in place of five:
//  - dq: as the forward pass, 128 pairs a workgroup, queries and dout in
//    registers, 64 keys a step through LDS.  It notes lse2 and delta for the other.
//  - dk and dv: 128 keys of a key/value head a workgroup, 32 a wave; the pairs
//    that see them pass through LDS, 32 a step, heads of a group side by side.
//    Scores stand the other way round here (pairs on the rows), so that weights
//    and score gradients are operands of the products over pairs in place.
//
// One sequence of 8,192 rows (32 heads on 8, D = 128, bf16): dq 840 to 910 us (930
// TFLOP/s of its three products; some of its scores' causal tests are branches, and
// the others are made in every step), dk and dv 1,190 to 1,280 us (850 to 920 of
// their four; the matrix units are busy 51 % of the cycles in which a CU has work,
// and 7 % of them it has none); with the forward pass 2,440 to 2,590 us.
#include <algorithm>
#include <atomic>

#include "prompt.hpp"

namespace ltk {

namespace {

template <int D>
constexpr int kTileBytes = 64 * D * 2;
template <int D>
constexpr int kStage = 2 * kTileBytes<D>;

__device__ __forceinline__ uint8_t* lds() {
    extern __shared__ at_u32x4 prompt_bwd_lds[];
    return reinterpret_cast<uint8_t*>(prompt_bwd_lds);
}

// log2(e) lse, infinite for a row that sees no key (its weights are 0 then).
__device__ __forceinline__ float base2(float lse) { return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f; }
// A row's two numbers as the dk and dv launch takes them: its weights come out
// 2^kUp times their size, and its score gradients as they are.
template <class E>
__device__ __forceinline__ void note_stats(const PromptArgs& a, int64_t row, float lse2, float delta) {
    a.lse2[row] = lse2 - E::kUp;
    a.delta[row] = delta * E::kDown;
}

// A lane's share of delta = dout . (out + rest): dimensions 16 j + 8 g ..; the
// lanes c and c + 32 of a wave share a row.
template <class E, int D>
__device__ __forceinline__ float delta_share(const PromptArgs& a, int64_t row, int g, const at_u32x4 (&dout)[D / 16]) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        const at_u32x4 y = *reinterpret_cast<const at_u32x4*>(a.out_in + row * D + 16 * j + 8 * g);
        at_u32x4 z{0u, 0u, 0u, 0u};
        if (a.rest_in) z = *reinterpret_cast<const at_u32x4*>(a.rest_in + row * D + 16 * j + 8 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = __builtin_fmaf(E::lo(dout[j][i]), E::lo(y[i]) + E::lo(z[i]), s);
            s = __builtin_fmaf(E::hi(dout[j][i]), E::hi(y[i]) + E::hi(z[i]), s);
        }
    }
    return s;
}

// lse2 and delta of every row and head, where no dq is asked for (its launch forms
// them too, in the same order).
template <class E, int D>
__global__ __launch_bounds__(64 * kWaves) void prompt_delta_kernel(PromptArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 31, g = lane >> 5;
    const int64_t r = (int64_t)blockIdx.x * kUnit + 32 * wave + c;
    float s = 0.0f;
    if (r < (int64_t)a.T * a.Hq) {
        const int t = (int)(r / a.Hq), h = (int)(r % a.Hq);
        at_u32x4 dout[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            dout[j] = *reinterpret_cast<const at_u32x4*>(a.dout.p + t * a.dout.row + h * a.dout.head + 16 * j + 8 * g);
        s = delta_share<E, D>(a, r, g, dout);
    }
    s = pr_sum_halves(s);
    if (r < (int64_t)a.T * a.Hq && g == 0) note_stats<E>(a, r, base2(a.lse[r]), s);
}

// dq: units are row tiles as in the forward pass.
template <class E, int D>
__global__ __launch_bounds__(64 * kWaves, 2) void prompt_dq_kernel(PromptArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, g = lane >> 5;
    const PrPlace pl = pr_place(a);
    const int h = pl.h;
    PrRowUnit u;
    if (!pr_row_unit(a, pl.unit, u)) return;
    const PrParts parts = pr_parts(a, u.t1 - u.t0);
    if (pl.part >= parts.used) return;
    const int t0 = u.t0 + pl.part * parts.size, t1 = min(t0 + parts.size, u.t1);
    const PrSeq& s = u.s;

    // the wave's rows
    const int fw = 32 * wave;
    const bool have = fw + c < u.count;
    const PrPair pr = pr_pair(a, u.first, fw + c);
    const int pos = have && s.in ? s.pos0() + pr.i : -1;
    const int64_t row = have ? (int64_t)(s.r0 + pr.i) * a.Hq + h * a.G + pr.g : -1;
    const int wlo = s.pos0() + pr_pair(a, u.first, fw).i, whi = s.pos0() + pr_pair(a, u.first, min(fw + 31, u.count - 1)).i;
    at_u32x4 q[D / 16], dout[D / 16];
    float lse2 = INFINITY, delta = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) q[j] = dout[j] = at_u32x4{0u, 0u, 0u, 0u};
    if (have && s.in) {
        const int64_t t = s.r0 + pr.i, x = h * a.G + pr.g;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            q[j] = *reinterpret_cast<const at_u32x4*>(a.q.p + t * a.q.row + x * a.q.head + 16 * j + 8 * g);
            dout[j] = *reinterpret_cast<const at_u32x4*>(a.dout.p + t * a.dout.row + x * a.dout.head + 16 * j + 8 * g);
        }
        delta = delta_share<E, D>(a, row, g, dout);
        lse2 = base2(a.lse[row]);
    }
    delta = pr_sum_halves(delta);
    if (have && pl.part == 0 && g == 0) note_stats<E>(a, row, lse2, delta);
    pr_f32x16 o[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[t][r] = 0.0f;
    const int from = a.window > 0 ? max(pos, 0) - a.window : -1;

    auto copy = [&](int t) {
        uint8_t* st = lds() + (t & 1) * kStage<D>;
        pr_copy_tile<D>(a.k, s.k0, h, t * kKeys, s.m, st);
        pr_copy_tile<D>(a.v, s.k0, h, t * kKeys, s.m, st + kTileBytes<D>);
    };
    const int along = pr_along<D>(), across = pr_across<D>();
    if (t0 < t1) copy(t0);
    pr_wait_copies();
    __syncthreads();
    if (fw >= u.count) {   // a wave without rows only copies
        for (int t = t0; t < t1; ++t) {
            if (t + 1 < t1) copy(t + 1);
            pr_wait_copies();
            __syncthreads();
        }
        return;
    }
    for (int t = t0; t < t1; ++t) {
        if (t + 1 < t1) copy(t + 1);
        const int stage = (t & 1) * kStage<D>, kt = pr_per_step(along) + stage, ka = pr_per_step(across) + stage;
        const int vt = kt + kTileBytes<D>;
        const int key0 = t * kKeys;
        const bool whole = key0 + kKeys - 1 <= wlo && (a.window <= 0 || key0 > whi - a.window);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            pr_f32x16 x, y;
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) x = E::mfma(pr_read<D>(lds(), kt, b, j), q[j], x);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) y = E::mfma(pr_read<D>(lds(), vt, b, j), dout[j], y);
            at_u32x4 ds[2];
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                float z[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float p = __builtin_fmaf(x[r + i], a.c2, -lse2);
                    const int key = key0 + 32 * b + 8 * (r / 4) + 4 * g + r % 4 + i;
                    if (!whole) p = (key <= pos) & (key > from) ? p : -INFINITY;
                    z[i] = __builtin_amdgcn_exp2f(p) * (y[r + i] - delta);
                }
                ds[r / 8][(r % 8) / 2] = E::pack(z[0], z[1]);
            }
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int t = 0; t < D / 32; ++t) o[t] = E::mfma(pr_read_across<D>(lds(), ka, 2 * b + w, t), ds[w], o[t]);
        }
        pr_wait_copies();
        __syncthreads();
    }
    if (row < 0) return;
    if (parts.used <= 1) {
        pr_store_row<E, D>(a.dq + row * D, g, o, a.scale);
        return;
    }
    float* part = a.part + ((pl.unit * a.Hkv + h) * a.splits + pl.part) * (int64_t)(kUnit * D);
    const int r = fw + c;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<at_f32x4*>(part + (size_t)r * D + 32 * t + 8 * i + 4 * g) =
                at_f32x4{o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
}

// Sums the parts of a unit's dq, 8 rows a workgroup.
template <class E, int D>
__global__ __launch_bounds__(2 * D) void prompt_dq_join_kernel(PromptArgs a) {
    const int64_t un = blockIdx.x / (uint32_t)a.Hkv;
    const int h = (int)(blockIdx.x - (uint32_t)un * (uint32_t)a.Hkv);
    PrRowUnit u;
    if (!pr_row_unit(a, un, u)) return;
    const int used = pr_parts(a, u.t1 - u.t0).used;
    if (used <= 1) return;
    const int r = blockIdx.y * 8 + threadIdx.x / (D / 4), d = 4 * (threadIdx.x % (D / 4));
    if (r >= u.count) return;
    const float* part = a.part + (un * a.Hkv + h) * a.splits * (int64_t)(kUnit * D) + (size_t)r * D + d;
    at_f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int i = 0; i < used; ++i) o += *reinterpret_cast<const at_f32x4*>(part + (int64_t)i * (kUnit * D));
    const PrPair p = pr_pair(a, u.first, r);
    const int64_t row = (int64_t)(u.s.r0 + p.i) * a.Hq + h * a.G + p.g;
    *reinterpret_cast<at_u32x2*>(a.dq + row * D + d) =
        at_u32x2{E::pack(o[0] * a.scale, o[1] * a.scale), E::pack(o[2] * a.scale, o[3] * a.scale)};
}

// LDS of the dk and dv kernel: the unit's rows of v, two stages, constants of the threads.
template <int D>
constexpr int kPairTile = kPairs * D * 2;
template <int D>
constexpr int kKvStage = 2 * kPairTile<D> + 2 * kPairs * 4;   // rows of q, of dout, then the pairs' lse2 and delta
template <int D>
constexpr int kStagesAt = kUnit * D * 2;
template <int D>
constexpr int kMineAt = kStagesAt<D> + 2 * kKvStage<D>;
template <int D>
constexpr int kKvLds = kMineAt<D> + 64 * kWaves * 16;

// Pairs [f0, f1) that may see keys [ka, kb) of a sequence.
__device__ __forceinline__ void seeing(const PromptArgs& a, const PrSeq& s, int ka, int kb, int64_t& f0, int64_t& f1) {
    const int pos0 = s.pos0();
    const int i0 = max(ka - pos0, 0);
    const int i1 = a.window > 0 ? (int)min((int64_t)s.n, (int64_t)kb - 1 + a.window - pos0) : s.n;
    f0 = (int64_t)i0 * a.G;
    f1 = s.in ? max((int64_t)i1 * a.G, f0) : f0;
}

// dk and dv: a unit is 128 keys of a key/value head, 32 a wave; the pairs that see
// them pass through LDS, 32 a step.  A wave keeps its rows of k and both sums in
// registers; those of v wait in LDS (with them in registers too, 25 and more of
// the 256 spilled, and each reload waited for all copies on their way: one
// sequence of 8,192 rows 1,587 us against 1,376, the vector work between the
// matrix instructions included, for which there were no registers either).
template <class E, int D>
__global__ __launch_bounds__(64 * kWaves, 2) void prompt_dkv_kernel(PromptArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, g = lane >> 5;
    const PrPlace pl = pr_place(a);
    const int h = pl.h, split = pl.part;
    const int64_t un = pl.unit;
    int64_t tile;   // (the first keys are seen by the most rows)
    const PrSeq s = pr_seq_of<kUnit, true>(a, un, 1, tile);
    if (tile * kUnit >= s.m) return;
    const int ka = (int)tile * kUnit, kb = min(ka + kUnit, s.m), pos0 = s.pos0();
    const int kw = ka + 32 * wave;
    int64_t f0, f1;
    seeing(a, s, ka, kb, f0, f1);
    const PrParts parts = pr_parts(a, uniform((int)((f1 - f0 + kPairs - 1) / kPairs)));
    if (split >= parts.used) return;
    f0 += (int64_t)split * parts.size * kPairs;
    f1 = min(f0 + (int64_t)parts.size * kPairs, f1);
    const int steps = uniform((int)((f1 - f0 + kPairs - 1) / kPairs));

    pr_f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) dk[t][r] = dv[t][r] = 0.0f;
    at_u32x4 kf[D / 16];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        kf[j] = at_u32x4{0u, 0u, 0u, 0u};
        if (kw + c < kb && s.in)
            kf[j] = *reinterpret_cast<const at_u32x4*>(a.k.p + (int64_t)(s.k0 + kw + c) * a.k.row + (int64_t)h * a.k.head +
                                                       16 * j + 8 * g);
    }

    PrPair at{uniform((int)((uint32_t)f0 / (uint32_t)a.G)), uniform((int)((uint32_t)f0 % (uint32_t)a.G))};   // a step's first pair
    // A copy of 1 KB takes kRowsPer pairs.  Where those are heads of one row, or
    // whole rows, a lane's place relative to the first of them never changes.
    constexpr int kRowsPer = 512 / D, kCopies = kPairs / kRowsPer / kWaves;
    const bool even = a.G % kRowsPer == 0 || kRowsPer % a.G == 0;
    const int lr = lane / (D / 8), li = a.G < kRowsPer ? lr / a.G : 0, lg = a.G < kRowsPer ? lr % a.G : lr;
    // What a thread needs once a step waits in LDS: the sums and k leave no
    // registers for it.
    at_u32x4* mine = reinterpret_cast<at_u32x4*>(lds() + kMineAt<D>) + threadIdx.x;
    *mine = at_u32x4{2u * ((uint32_t)li * (uint32_t)a.q.row + (uint32_t)lg * (uint32_t)a.q.head),
                     2u * ((uint32_t)li * (uint32_t)a.dout.row + (uint32_t)lg * (uint32_t)a.dout.head),
                     ((lane % (D / 8)) ^ pr_swizzle<D>(lr)) * 16u, (uint32_t)(pr_along<D>() | pr_across<D>() << 16)};
    auto copy = [&](int t, const at_u32x4& my) {   // of the step that begins at `at`
        uint8_t* st = lds() + kStagesAt<D> + (t & 1) * kKvStage<D>;
        const int left = (int)min(f1 - f0 - (int64_t)t * kPairs, (int64_t)kPairs);   // pairs of the step
        if (even && left == kPairs) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int r0 = (wave * kCopies + i) * kRowsPer;
                const PrPair p = pr_pair(a, at, r0);
                const int64_t y = s.r0 + p.i, x = h * a.G + p.g;
                // (the swizzle of row r0 + lr is that of row lr but for two bits)
                const uint32_t chunk = my[2] ^ (uint32_t)(16 * pr_swizzle<D>(r0));
                lds_direct16_async(a.q.p + y * a.q.row + x * a.q.head, my[0] + chunk, st + r0 * (2 * D));
                lds_direct16_async(a.dout.p + y * a.dout.row + x * a.dout.head, my[1] + chunk, st + kPairTile<D> + r0 * (2 * D));
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kCopies; ++i) {
                const int ln = pr_per_step(lane), r0 = (wave * kCopies + i) * kRowsPer, r = r0 + ln / (D / 8);
                const int chunk = (ln % (D / 8)) ^ pr_swizzle<D>(r);
                const PrPair p = pr_pair(a, at, min(r, left - 1));
                const int64_t y = s.r0 + p.i, x = h * a.G + p.g;
                lds_direct16_async(a.q.p + y * a.q.row + x * a.q.head + 8 * chunk, st + r0 * (2 * D));
                lds_direct16_async(a.dout.p + y * a.dout.row + x * a.dout.head + 8 * chunk, st + kPairTile<D> + r0 * (2 * D));
            }
        }
        if (wave == 0) {   // (uniform) lse2 by the first half of the lanes, delta by the others
            const int ln = pr_per_step(lane);
            const PrPair p = pr_pair(a, at, min(ln & 31, left - 1));
            const float* src = ln < 32 ? a.lse2 : a.delta;
            lds_direct4_async(src + (int64_t)(s.r0 + p.i) * a.Hq + h * a.G + p.g, st + 2 * kPairTile<D>);
        }
    };
    // (a scale of 0 is taken as the least one, so that a hidden score stays infinite)
    const float c2 = a.c2 == 0.0f ? 0x1p-126f : a.c2;
    if (steps > 0) {
        pr_copy_tile<D>(a.v, s.k0, h, ka, s.m, lds());
        pr_copy_tile<D>(a.v, s.k0, h, min(ka + 64, s.m - 1), s.m, lds() + kTileBytes<D>);
        copy(0, *mine);
    }
    pr_wait_copies();
    __syncthreads();
    for (int t = 0; t < steps; ++t) {
        const PrPair now = at;
        const int left = (int)min(f1 - f0 - (int64_t)t * kPairs, (int64_t)kPairs);
        const int plo = pos0 + now.i, phi = pos0 + uniform(pr_pair(a, now, left - 1).i);
        const bool whole = kw + 31 <= plo && left == kPairs && (a.window <= 0 || kw > phi - a.window);
        const PrPair next = pr_pair(a, at, kPairs);
        at = PrPair{uniform(next.i), uniform(next.g)};
        const at_u32x4 my = *mine;
        const int along = my[3] & 0xffff, across = my[3] >> 16;
        if (t + 1 < steps) copy(t + 1, my);
        const int stage = kStagesAt<D> + (t & 1) * kKvStage<D>;
        const float* stat = reinterpret_cast<const float*>(lds() + stage + 2 * kPairTile<D>) + 4 * g;

        // N matrix instructions each: scores, dout v, dv, dk.  The weights are formed
        // between those of dout v, the score gradients between those of dv; what they
        // read from LDS is read kAhead of them before.
        constexpr int N = D / 16, kAhead = 4, kNear = 2;
        at_u32x4 frag[kAhead], vfrag[kNear];
        at_f32x2 sf[kNear];
        int place = 0, vplace = 0;
        auto fetch = [&](int n) {
            if (n >= 4 * N) return;
            const int k = n / N, j = n % N;
            if (j == 0) place = pr_per_step(k < 2 ? along : across) + stage + (k == 1 || k == 2 ? kPairTile<D> : 0);
            frag[n % kAhead] = k < 2 ? pr_read<D>(lds(), place, 0, j) : pr_read_across<D>(lds(), place, j / (D / 32), j % (D / 32));
        };
        auto fetch_v = [&](int j) {
            if (j < 0 || j >= N) return;
            if (j == 0) vplace = pr_per_step(along) + wave * (64 * D);
            vfrag[j % kNear] = pr_read<D>(lds(), vplace, 0, j);
        };
        // lse2, then delta, of scores 2 i and 2 i + 1
        auto fetch_stat = [&](int i) {
            if (i < 16) sf[i % kNear] = *reinterpret_cast<const at_f32x2*>(stat + (i / 8) * kPairs + 8 * (i % 8 / 2) + 2 * (i % 2));
        };
        auto less_delta = [](float dp, float delta) {   // (the factor is a power of two: dp - delta, rounded, times it)
            return E::kUp == 0.0f ? dp - delta : __builtin_fmaf(dp, E::kDown, -delta);
        };
        pr_f32x16 x, y;
        at_u32x4 pf[2], ds[2];
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x = E::mfma(frag[j % kAhead], kf[j], x);
            fetch(j + kAhead);
            fetch_v(j - (N - kNear));
            if (j >= N - kNear) fetch_stat(j - (N - kNear));
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!whole) {   // hidden pairs' scores: to weights of 0
            const int ln = pr_per_step(lane), first = 4 * (ln >> 5), key = kw + (ln & 31);
            const float hidden = c2 > 0.0f ? -INFINITY : INFINITY;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int f = first + 8 * (r / 4) + r % 4, pos = pos0 + pr_pair(a, now, f).i;
                const int from = a.window > 0 ? max(pos, 0) - a.window : -1;
                x[r] = (f < left) & (key <= pos) & (key > from) ? x[r] : hidden;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            y = E::mfma(frag[j % kAhead], vfrag[j % kNear], y);
            fetch(N + j + kAhead);
            fetch_v(j + kNear);
#pragma unroll
            for (int i = 8 / N * j; i < 8 / N * (j + 1); ++i) {
                x[2 * i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * i], c2, -sf[i % kNear][0]));
                x[2 * i + 1] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * i + 1], c2, -sf[i % kNear][1]));
                pf[i / 4][i % 4] = E::pack(x[2 * i], x[2 * i + 1]);
                fetch_stat(i + kNear);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            dv[j % (D / 32)] = E::mfma(frag[j % kAhead], pf[j / (D / 32)], dv[j % (D / 32)]);
            fetch(2 * N + j + kAhead);
#pragma unroll
            for (int i = 8 / N * j; i < 8 / N * (j + 1); ++i) {
                const float z0 = less_delta(y[2 * i], sf[i % kNear][0]), z1 = less_delta(y[2 * i + 1], sf[i % kNear][1]);
                ds[i / 4][i % 4] = E::pack(x[2 * i] * z0, x[2 * i + 1] * z1);
                fetch_stat(8 + i + kNear);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            dk[j % (D / 32)] = E::mfma(frag[j % kAhead], ds[j / (D / 32)], dk[j % (D / 32)]);
            fetch(3 * N + j + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
        pr_wait_copies();
        __syncthreads();
    }
    const int key = kw + c;
    if (key >= kb) return;
    if (parts.used <= 1) {
        const int64_t row = (int64_t)(s.k0 + key) * a.Hkv + h;
        pr_store_row<E, D>(a.dk + row * D, g, dk, a.scale);
        pr_store_row<E, D>(a.dv + row * D, g, dv, E::kDown);
        return;
    }
    // a part: 128 keys' dk, then their dv
    float* part = a.part + ((un * a.Hkv + h) * a.splits + split) * (int64_t)(2 * kUnit * D) + (size_t)(32 * wave + c) * D;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<at_f32x4*>(part + 32 * t + 8 * i + 4 * g) =
                at_f32x4{dk[t][4 * i], dk[t][4 * i + 1], dk[t][4 * i + 2], dk[t][4 * i + 3]};
            *reinterpret_cast<at_f32x4*>(part + (size_t)kUnit * D + 32 * t + 8 * i + 4 * g) =
                at_f32x4{dv[t][4 * i], dv[t][4 * i + 1], dv[t][4 * i + 2], dv[t][4 * i + 3]};
        }
}

// Sums the parts of a unit's dk and dv, 8 keys a workgroup.
template <class E, int D>
__global__ __launch_bounds__(2 * D) void prompt_dkv_join_kernel(PromptArgs a) {
    const int64_t un = blockIdx.x / (uint32_t)a.Hkv;
    const int h = (int)(blockIdx.x - (uint32_t)un * (uint32_t)a.Hkv);
    int64_t tile;   // (the first keys are seen by the most rows)
    const PrSeq s = pr_seq_of<kUnit, true>(a, un, 1, tile);
    if (tile * kUnit >= s.m) return;
    const int ka = (int)tile * kUnit, kb = min(ka + kUnit, s.m);
    int64_t f0, f1;
    seeing(a, s, ka, kb, f0, f1);
    const int used = pr_parts(a, (int)((f1 - f0 + kPairs - 1) / kPairs)).used;
    if (used <= 1) return;
    const int r = blockIdx.y * 8 + threadIdx.x / (D / 4), d = 4 * (threadIdx.x % (D / 4));
    if (ka + r >= kb) return;
    const float* part = a.part + (un * a.Hkv + h) * a.splits * (int64_t)(2 * kUnit * D) + (size_t)r * D + d;
    at_f32x4 x{0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll 4
    for (int i = 0; i < used; ++i, part += 2 * kUnit * D) {
        x += *reinterpret_cast<const at_f32x4*>(part);
        y += *reinterpret_cast<const at_f32x4*>(part + (size_t)kUnit * D);
    }
    const int64_t row = (int64_t)(s.k0 + ka + r) * a.Hkv + h;
    *reinterpret_cast<at_u32x2*>(a.dk + row * D + d) =
        at_u32x2{E::pack(x[0] * a.scale, x[1] * a.scale), E::pack(x[2] * a.scale, x[3] * a.scale)};
    y *= E::kDown;
    *reinterpret_cast<at_u32x2*>(a.dv + row * D + d) = at_u32x2{E::pack(y[0], y[1]), E::pack(y[2], y[3])};
}

// More than 64 KB of LDS is asked for once per device.
template <class F>
hipError_t allow_lds(F* kernel, int bytes, std::atomic<uint64_t>& allowed) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) & bit)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    return hipSuccess;
}

template <class E, int D>
hipError_t launch(const PromptPlan& p, PromptArgs& a, hipStream_t st) {
    const int64_t rows = (int64_t)a.T * a.Hq;
    if (!a.dq && rows > 0) prompt_delta_kernel<E, D><<<(unsigned)((rows + kUnit - 1) / kUnit), 64 * kWaves, 0, st>>>(a);
    if (a.dq && rows > 0) {
        a.splits = p.grad.splits, a.per = p.grad.per, a.units = p.grad.units;
        prompt_dq_kernel<E, D><<<(unsigned)p.grad.blocks, 64 * kWaves, 2 * kStage<D>, st>>>(a);
        if (a.splits > 1)
            prompt_dq_join_kernel<E, D><<<dim3((unsigned)(a.units * a.Hkv), kUnit / 8), 2 * D, 0, st>>>(a);
    }
    if (a.dk && a.S > 0) {
        a.splits = p.keys.splits, a.per = p.keys.per, a.units = p.keys.units;
        if constexpr (kKvLds<D> > 65536) {
            static std::atomic<uint64_t> allowed;
            const hipError_t e = allow_lds(prompt_dkv_kernel<E, D>, kKvLds<D>, allowed);
            if (e != hipSuccess) return e;
        }
        prompt_dkv_kernel<E, D><<<(unsigned)p.keys.blocks, 64 * kWaves, kKvLds<D>, st>>>(a);
        if (a.splits > 1)
            prompt_dkv_join_kernel<E, D><<<dim3((unsigned)(a.units * a.Hkv), kUnit / 8), 2 * D, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_prompt_backward(const PromptPlan& p, int type, int D, PromptArgs& a, void* ws, hipStream_t st) {
    a.lse2 = static_cast<float*>(ws);
    a.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.stat_bytes);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 2 * p.stat_bytes);
    if (type == LTK_ROWS_BF16) return D == 64 ? launch<PrBf16, 64>(p, a, st) : launch<PrBf16, 128>(p, a, st);
    return D == 64 ? launch<PrF16, 64>(p, a, st) : launch<PrF16, 128>(p, a, st);
}

}  // namespace ltk
