// prompt.hip -- causal attention over packed 16-bit prompts on gfx950: bound by
// the matrix cores and the exponentials beside them.
//
//   y_s = scale log2(e) (q . k_s),  out = sum 2^(y_s - m) v_s / l,
//   l = sum 2^(y_s - m),  lse = ln(2) (m + log2 l),
// one pass with a running reference m that moves only where a score passes it by
// 8 (kSlack): most steps need no exchange between lanes and scale nothing.  In fp16
// m lies 7 below the score that it moved to (kLift).
//
// A workgroup of four waves takes 128 (row, head) pairs of one key/value head,
// 32 a wave, and 64 keys a step.  The query heads that share a key/value head lie
// side by side among the pairs, so keys are read once for all of them, and with
// several heads a group the border of the causal mask costs little (16 rows a
// tile for groups of eight).
//  - Scores are formed transposed (keys on the rows of v_mfma_f32_32x32x16, pairs
//    on its columns; the wave's queries stay in registers): a lane holds one
//    pair's scores against 16 keys, which is the layout that the second product
//    wants for its weights.  Those are rounded once to 16 bits in place (2^-8 of
//    themselves in bf16: the second product takes operands of one type, and the
//    values are bf16).
//  - Keys and values go from memory to LDS without passing through registers, as
//    they lie; the second product's operands across rows are read with the
//    transposing LDS read.  Both reads are free of bank conflicts (pr_swizzle).
//  - Keys have two stages and values one, 48 KB at D = 128, so that three
//    workgroups run on a CU: while one forms exponentials, another feeds the
//    matrix unit.  A step's values are on their way while its scores are formed,
//    the next keys during all of it.  (Both in two stages, two workgroups: one
//    sequence of 16,384 rows 4,450 us against 4,105.)
//
// One sequence of 16,384 rows (64 heads on 8, D = 128, bf16: 4.4e12 operations)
// takes 4,080 to 4,380 us, 1,000 to 1,080 TFLOP/s of the 1,207 that a large matrix
// product reaches: the matrix units are busy 56 % of the cycles, the vector units
// 57 %.  The causal test costs every step something, where no key is hidden too: it
// is compiled to a scalar branch for each of a lane's 32 scores, and nothing moves
// between them.  16 prompts of up to 2,039 rows (32 on 8) take 224 to 246 us, 690 to 760
// TFLOP/s: units are 11 steps long on average, and finding the unit, its first
// tile and its stores take 14 % of a unit's time.  Two of up to 8,111 with a
// window of 1,024 (D = 64, fp16) take 155 to 166 us, 670 to 710 TFLOP/s: half the
// products for the same exponentials and branches.  The smallest calls take 6 us:
// launch, offsets, tile.
#include <math.h>

#include <algorithm>

#include "prompt.hpp"

namespace ltk {

namespace {

template <int D>
constexpr int kTileBytes = kKeys * D * 2;

__device__ __forceinline__ uint8_t* lds() {
    extern __shared__ at_u32x4 prompt_lds[];
    return reinterpret_cast<uint8_t*>(prompt_lds);
}

template <class E, int D>
__global__ __launch_bounds__(64 * kWaves, 3) void prompt_kernel(PromptArgs a) {
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
    at_u32x4 q[D / 16];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        q[j] = at_u32x4{0u, 0u, 0u, 0u};
        if (have && s.in)
            q[j] = *reinterpret_cast<const at_u32x4*>(a.q.p + (int64_t)(s.r0 + pr.i) * a.q.row +
                                                      (int64_t)(h * a.G + pr.g) * a.q.head + 16 * j + 8 * g);
    }
    float m = 0.0f, over = -INFINITY, l = 0.0f;
    pr_f32x16 o[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[t][r] = 0.0f;
    const int from = a.window > 0 ? max(pos, 0) - a.window : -1;

    auto copy_keys = [&](int t) { pr_copy_tile<D>(a.k, s.k0, h, t * kKeys, s.m, lds() + (t & 1) * kTileBytes<D>); };
    auto copy_values = [&](int t) { pr_copy_tile<D>(a.v, s.k0, h, t * kKeys, s.m, lds() + 2 * kTileBytes<D>); };
    const int along = pr_along<D>(), across = pr_across<D>();
    if (t0 < t1) {
        copy_keys(t0);
        copy_values(t0);
    }
    pr_wait_copies();
    __syncthreads();
    if (fw >= u.count) {   // a wave without rows only copies (as often as the others wait for each other)
        for (int t = t0; t < t1; ++t) {
            if (t + 1 < t1) copy_keys(t + 1);
            if (t + 1 < t1)
                pr_wait_copies_but<D / 8 / kWaves>();
            else
                pr_wait_copies();
            __syncthreads();
            pr_wait_copies();
            __syncthreads();
            if (t + 1 < t1) copy_values(t + 1);
        }
        return;
    }
    for (int t = t0; t < t1; ++t) {
        if (t + 1 < t1) copy_keys(t + 1);
        const int kt = pr_per_step(along) + (t & 1) * kTileBytes<D>, vt = pr_per_step(across) + 2 * kTileBytes<D>;
        const int key0 = t * kKeys;
        pr_f32x16 x[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int r = 0; r < 16; ++r) x[b][r] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) x[b] = E::mfma(pr_read<D>(lds(), kt, b, j), q[j], x[b]);
        }
        const bool whole = key0 + kKeys - 1 <= wlo && (a.window <= 0 || key0 > whi - a.window);
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float y = __builtin_fmaf(x[b][r], a.c2, -m);
                const int key = key0 + 32 * b + 8 * (r / 4) + 4 * g + r % 4;
                if (!whole) y = (key <= pos) & (key > from) ? y : -INFINITY;
                x[b][r] = y;
                top = fmaxf(top, y);
            }
        if (__ballot(top > over) != 0) {
            const float up = pr_max_halves(top);
            const bool move = up > over;
            const float d = move ? up - E::kLift : 0.0f;
            const float f = over == E::kLift + kSlack ? __builtin_amdgcn_exp2f(-d) : 1.0f;
            m += d;
            over = move ? E::kLift + kSlack : over;
            l *= f;
#pragma unroll
            for (int t = 0; t < D / 32; ++t) o[t] *= f;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) x[b][r] -= d;
        }
        at_u32x4 p[4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                const float p0 = __builtin_amdgcn_exp2f(x[b][r]), p1 = __builtin_amdgcn_exp2f(x[b][r + 1]);
                l += p0;
                l += p1;
                p[2 * b + r / 8][(r % 8) / 2] = E::pack(p0, p1);
            }
        // the values' copies are older than the next keys'
        if (t + 1 < t1)
            pr_wait_copies_but<D / 8 / kWaves>();
        else
            pr_wait_copies();
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int t = 0; t < D / 32; ++t) o[t] = E::mfma(pr_read_across<D>(lds(), vt, w, t), p[w], o[t]);
        pr_wait_copies();
        __syncthreads();
        if (t + 1 < t1) copy_values(t + 1);
    }
    l = pr_sum_halves(l);
    if (row < 0) return;
    if (parts.used <= 1) {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        pr_store_row<E, D>(a.out + row * D, g, o, inv);
        if (a.rest) {
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; i += 8)
                    pr_store16(a.rest + row * D + 32 * t + 2 * i, g, pr_rest<E>(o[t][i] * inv, o[t][i + 1] * inv),
                               pr_rest<E>(o[t][i + 2] * inv, o[t][i + 3] * inv), pr_rest<E>(o[t][i + 4] * inv, o[t][i + 5] * inv),
                               pr_rest<E>(o[t][i + 6] * inv, o[t][i + 7] * inv));
        }
        if (a.lse && g == 0) a.lse[row] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f : -INFINITY;
        return;
    }
    // a part: kUnit rows of D sums, then kUnit pairs (m, l)
    float* part = a.part + ((pl.unit * a.Hkv + h) * a.splits + pl.part) * (int64_t)(kUnit * (D + 2));
    const int r = fw + c;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<at_f32x4*>(part + (size_t)r * D + 32 * t + 8 * i + 4 * g) =
                at_f32x4{o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
    if (g == 0) {
        part[(size_t)kUnit * D + 2 * r] = l > 0.0f ? m : kNoRef;
        part[(size_t)kUnit * D + 2 * r + 1] = l;
    }
}

// Joins the parts of a unit, 8 rows a workgroup.
template <class E, int D>
__global__ __launch_bounds__(2 * D) void prompt_join_kernel(PromptArgs a) {
    const int64_t un = blockIdx.x / (uint32_t)a.Hkv;
    const int h = (int)(blockIdx.x - (uint32_t)un * (uint32_t)a.Hkv);
    PrRowUnit u;
    if (!pr_row_unit(a, un, u)) return;
    const int used = pr_parts(a, u.t1 - u.t0).used;
    if (used <= 1) return;
    const int r = blockIdx.y * 8 + threadIdx.x / (D / 4), d = 4 * (threadIdx.x % (D / 4));
    if (r >= u.count) return;
    const float* part = a.part + (un * a.Hkv + h) * a.splits * (int64_t)(kUnit * (D + 2));
    float m = kNoRef, l = 0.0f;
    at_f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int i = 0; i < used; ++i) m = fmaxf(m, part[(int64_t)i * (kUnit * (D + 2)) + (size_t)kUnit * D + 2 * r]);
#pragma unroll 8
    for (int i = 0; i < used; ++i, part += kUnit * (D + 2)) {
        const float f = __builtin_amdgcn_exp2f(part[(size_t)kUnit * D + 2 * r] - m);
        l = __builtin_fmaf(f, part[(size_t)kUnit * D + 2 * r + 1], l);
        o += *reinterpret_cast<const at_f32x4*>(part + (size_t)r * D + d) * f;
    }
    const PrPair p = pr_pair(a, u.first, r);
    const int64_t row = (int64_t)(u.s.r0 + p.i) * a.Hq + h * a.G + p.g;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    o *= inv;
    *reinterpret_cast<at_u32x2*>(a.out + row * D + d) = at_u32x2{E::pack(o[0], o[1]), E::pack(o[2], o[3])};
    if (a.rest)
        *reinterpret_cast<at_u32x2*>(a.rest + row * D + d) = at_u32x2{pr_rest<E>(o[0], o[1]), pr_rest<E>(o[2], o[3])};
    if (a.lse && d == 0) a.lse[row] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f : -INFINITY;
}

template <class E, int D>
hipError_t launch(const PromptPlan& p, const PromptArgs& a, hipStream_t st) {
    prompt_kernel<E, D><<<(unsigned)p.rows.blocks, 64 * kWaves, 3 * kTileBytes<D>, st>>>(a);
    if (a.splits > 1)
        prompt_join_kernel<E, D><<<dim3((unsigned)(p.rows.units * a.Hkv), 4 * kWaves), 2 * D, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

// Units are cut while there are too few of them for the card to run evenly: the
// units of one sequence differ in length by up to the whole of it, so that with
// more than one for each of the `places` workgroups that run at once the short
// ones fill up what the long ones leave.  Below that, a part is about what a
// place has to do.  `units` are about those with rows, `mean` the steps of one in
// a sequence of average length, `most` those in a sequence that is all of the
// batch.  The parts pass through memory and the joining launch costs some steps'
// time: parts have `least` steps or more, but for a unit's last one, and cutting
// has to take that many off the longest unit (about the geometric mean of twice
// the mean and the most).
// (Forward, 32 heads on 8, D = 128: 1,024 units for the 768 places 180 us whole
// and 197 cut, four prompts of 1,024 rows 57 whole and 84 cut, one of 2,048, 512
// units, 72 cut; a step of 8,192 rows 3,065 us with dk and dv whole, 2,510 cut.
// 64 heads on 8, 1,000 rows: dq's 500 units of 16 steps or less cut cost the step
// 12 us of 177.)
//
// The rule goes by totals, which is all that the host knows, so it does not see one
// sequence that is far longer than all others: its units stay whole where the others
// make enough units, and there are few parts a unit where they make many.  (One row
// each, 32 heads on 8, D = 128: 250 sequences, one of 65,536 keys and the others of
// 500, 2,360 us, 250 of as many keys in all 153; 128 such, 840 and 136.  A training
// step of 100 sequences of 256 rows beside one of 8,192: 3,550 us, the long one alone
// 2,420.)
static PromptCut cut(int64_t all, double units, double mean, int64_t most, int Hkv, int64_t places, int64_t least) {
    PromptCut c{all, all * Hkv, 1, 1 << 30};
    const int64_t per = std::max(least, (int64_t)(1.1 * units * Hkv * mean / places) + 1);
    if (units * Hkv >= 1.25 * places || sqrt(2.0 * mean * most) < per + least) return c;
    c.splits = (int)std::min((most + per - 1) / per, 3 * places / c.blocks + 1);
    c.per = (int)per;
    c.blocks *= c.splits;
    return c;
}

// Mean of min(x, cap) over lo <= x <= hi.
static double mean_capped(double lo, double hi, double cap) {
    if (cap >= hi) return 0.5 * (lo + hi);
    if (cap <= lo) return cap;
    return (0.5 * (cap * cap - lo * lo) + cap * (hi - cap)) / (hi - lo);
}

PromptPlan prompt_plan(int T, int S, int Hq, int Hkv, int D, int n_seq, int window) {
    PromptPlan p{};
    const int64_t G = Hq / Hkv, seqs = std::max(n_seq, 1);
    const double n = (double)T / seqs, m = (double)S / seqs, reach = window > 0 ? (double)window + kUnit : (double)S + kUnit;
    // (about: a sequence's last unit is half full)
    const int64_t row_units = pr_units(T, G, kUnit, n_seq), key_units = pr_units(S, 1, kUnit, n_seq);
    const double row_about = (double)T * G / kUnit + 0.5 * seqs, key_about = (double)S / kUnit + 0.5 * seqs;
    const double uneven = n_seq > 1 ? 1.2 : 1.0;   // (of unequal sequences the long ones have most of the steps)
    const double row_mean = uneven * mean_capped(std::max(m - n, 0.0), m, reach) / kKeys + 0.5;
    const double key_mean = uneven * mean_capped(0.0, m, std::min(n, reach)) * G / kPairs + 0.5;
    const int64_t row_most = (int64_t)std::min((double)S, reach) / kKeys + 1, key_most = (int64_t)(std::min((double)T, reach) * G / kPairs) + 1;
    // workgroups that a CU holds, by registers and LDS: three of the forward pass,
    // two of the others at D = 128; at D = 64 four, three and two
    p.rows = cut(row_units, row_about, row_mean, row_most, Hkv, D == 64 ? 1024 : 768, 8);
    p.grad = cut(row_units, row_about, row_mean, row_most, Hkv, D == 64 ? 768 : 512, 8);
    p.keys = cut(key_units, key_about, key_mean, key_most, Hkv, 512, 16);
    auto parts = [&](const PromptCut& c, int64_t floats) { return c.splits > 1 ? (size_t)(c.blocks * kUnit * floats) * 4 : 0; };
    p.fwd_bytes = std::max<size_t>(256, parts(p.rows, D + 2));
    p.stat_bytes = ((size_t)T * Hq * 4 + 255) / 256 * 256;
    p.bwd_bytes = std::max<size_t>(256, 2 * p.stat_bytes + std::max(parts(p.grad, D), parts(p.keys, 2 * D)));
    // (the last: delta's launch)
    p.fits = grid_fits(std::max({p.rows.blocks, p.grad.blocks, p.keys.blocks, ((int64_t)T * Hq + kUnit - 1) / kUnit}), 64 * kWaves);
    return p;
}

hipError_t launch_prompt(const PromptPlan& p, int type, int D, PromptArgs& a, void* ws, hipStream_t st) {
    a.splits = p.rows.splits, a.per = p.rows.per, a.units = p.rows.units;
    a.part = static_cast<float*>(ws);
    if (type == LTK_ROWS_BF16) return D == 64 ? launch<PrBf16, 64>(p, a, st) : launch<PrBf16, 128>(p, a, st);
    return D == 64 ? launch<PrF16, 64>(p, a, st) : launch<PrF16, 128>(p, a, st);
}

}  // namespace ltk
