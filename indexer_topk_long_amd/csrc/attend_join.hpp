// attend_join.hpp -- units whose keys several workgroups share: how their
// partial rows lie in the workspace, and the launch that joins them.
//
// A part is fp32: RT rows of D accumulators, then RT pairs (m, l), for the
// weights 2^(y - m) that l and the accumulators are sums of.  Parts join as
//   m = max m_i,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m),
// always in the same order, so results do not depend on which workgroup ends
// first.
#pragma once

#include "attend.hpp"

namespace ltk {

namespace {

template <int D, int RT>
constexpr int part_floats() {
    return RT * (D + 2);
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

// A unit cut over n > 1 workgroups, as each of them notes it in the workspace
// for the join: [0] where it takes a later part of the unit (at the start of
// its range), [1] where it takes the first (at its end).  The parts are in the
// first one's slot, then in the slots 2 w of the workgroups w behind it.
struct Crossing {
    int n, i;           // parts (0: none), and which of them is this workgroup's
    int slot, behind;   // slot of the first part, and the workgroup of the second
    UnitRows u;
};
constexpr size_t crossing_bytes(int64_t blocks) { return (2 * sizeof(Crossing) * (size_t)blocks + 255) / 256 * 256; }

constexpr int kJoinRows = 8;   // lane groups (D / 4 lanes, a row's dimensions) of a joining workgroup

struct RowSum {
    float m, l;
    at_f32x4 o;
};
__device__ __forceinline__ void add_part(RowSum& s, float m, float l, const at_f32x4& o) {
    const bool up = m > s.m;   // the sum so far is scaled, else the part
    const Factor by(up ? s.m - m : m - s.m);
    s.l = up ? by.divisor(s.l) + l : s.l + by.divisor(l);
    s.o = s.o * (up ? by.f : 1.0f) + o * (up ? 1.0f : by.f);
    s.m = up ? m : s.m;
}
// Parts i0, i0 + step, .. below n of row `at` of a unit: part i at slot0
// (i == 0) or slot1 + (i - 1) slot_step.
template <int D, int RT>
__device__ __forceinline__ RowSum sum_parts(const AttendArgs& a, int at, int i0, int step, int n, int64_t slot0,
                                            int64_t slot1, int slot_step) {
    const int lane = threadIdx.x % (D / 4);
    RowSum s{kNoRef, 0.0f, at_f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll 4
    for (int i = i0; i < n; i += step) {
        const float* p = a.part + (i == 0 ? slot0 : slot1 + (int64_t)(i - 1) * slot_step) * part_floats<D, RT>();
        add_part(s, p[RT * D + at * 2], p[RT * D + at * 2 + 1],
                 *reinterpret_cast<const at_f32x4*>(p + at * D + 4 * lane));
    }
    return s;
}
template <int D, int PART>
__device__ __forceinline__ void write_row(const AttendArgs& a, int64_t row, const RowSum& s) {
    if constexpr (PART == kSharedKeys) {
        float* p = a.prior + row * (D + kPriorTail);
        const int d = 4 * (threadIdx.x % (D / 4));
        *reinterpret_cast<at_f32x4*>(p + d) = s.o;
        if (d == 0) p[D] = s.m, p[D + 1] = s.l;
        return;
    }
    const float inv = s.l > 0.0f ? 1.0f / s.l : 0.0f;
    *reinterpret_cast<at_u32x2*>(a.out + row * D + 4 * (threadIdx.x % (D / 4))) =
        at_u32x2{pack_bf16(s.o[0] * inv, s.o[1] * inv), pack_bf16(s.o[2] * inv, s.o[3] * inv)};
}
// One row by all lane groups, each every kJoinRows-th part.
template <int D, int RT, int PART = kAllKeys>
__device__ __forceinline__ void join_wide(const AttendArgs& a, int64_t row, int at, int n, int64_t slot0, int64_t slot1,
                                          int slot_step) {
    __shared__ float s_ml[kJoinRows][2];
    __shared__ float s_o[kJoinRows][D + 4];
    const int grp = threadIdx.x / (D / 4), lane = threadIdx.x % (D / 4);
    const RowSum s = sum_parts<D, RT>(a, at, grp, kJoinRows, n, slot0, slot1, slot_step);
    __syncthreads();
    *reinterpret_cast<at_f32x4*>(&s_o[grp][4 * lane]) = s.o;
    if (lane == 0) s_ml[grp][0] = s.m, s_ml[grp][1] = s.l;
    __syncthreads();
    if (grp != 0 || row < 0) return;
    RowSum all{kNoRef, 0.0f, at_f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int w = 0; w < kJoinRows; ++w) all.m = fmaxf(all.m, s_ml[w][0]);
#pragma unroll
    for (int w = 0; w < kJoinRows; ++w) {
        const Factor by(s_ml[w][0] - all.m);
        all.l += by.divisor(s_ml[w][1]);
        all.o += *reinterpret_cast<const at_f32x4*>(&s_o[w][4 * lane]) * by.f;
    }
    write_row<D, PART>(a, row, all);
}

// The workgroups (w, 0 .. join_hands<RT>() - 1) stand for workgroup w of the
// main launch: those of a cut unit's n workgroups share its rows, so that many
// parts have many hands, and those of uncut units end at once.  (Where nothing
// was cut, 8,192 workgroups of 128 threads took 12 us to end, 2,048 4 us.)
template <int RT>
constexpr int join_hands() {
    return RT > 64 ? RT / 32 : RT / kJoinRows;
}
template <int D, int RT, int PART>
__global__ __launch_bounds__(kJoinRows * D / 4) void attend_join_kernel(AttendArgs a) {
    const int grp = threadIdx.x / (D / 4);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const Crossing x = reinterpret_cast<const Crossing*>(a.head)[2 * (int64_t)blockIdx.x + e];
        if (x.n <= 1) continue;
        const int id = x.i * join_hands<RT>() + blockIdx.y, ids = x.n * join_hands<RT>();
        const int r0 = (int)((int64_t)id * RT / ids), r1 = (int)((int64_t)(id + 1) * RT / ids);
        const int64_t slot1 = 2 * (int64_t)x.behind;
        if (x.n < kJoinRows) {   // a row to a lane group
            for (int at = r0 + grp; at < r1; at += kJoinRows) {
                const int64_t row = out_row(a, x.u, x.u.f0 + at);
                if (row >= 0) write_row<D, PART>(a, row, sum_parts<D, RT>(a, at, 0, 1, x.n, x.slot, slot1, 2));
            }
        } else {
            for (int at = r0; at < r1; ++at)
                join_wide<D, RT, PART>(a, out_row(a, x.u, x.u.f0 + at), at, x.n, x.slot, slot1, 2);
        }
    }
}
template <int D, int RT, int PART>
void launch_join(const AttendPlan& p, const AttendArgs& a, hipStream_t st) {
    attend_join_kernel<D, RT, PART><<<dim3((unsigned)p.blocks, join_hands<RT>()), kJoinRows * D / 4, 0, st>>>(a);
}

}  // namespace

}  // namespace ltk
