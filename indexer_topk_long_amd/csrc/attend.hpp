// attend.hpp -- what the kernels of the paged e4m3 cache share: the cache and
// batch as kernels see them, the row and page lookups, and small conversions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "litetopk_attend.h"

namespace ltk {

typedef unsigned int at_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int at_u32x2 __attribute__((ext_vector_type(2)));
typedef float at_f32x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 at_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 at_bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 at_f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 at_f16x8 __attribute__((ext_vector_type(8)));

constexpr float kE4m3Max = 448.0f;

struct KvCache {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int n_pages, Hkv, page_shift;   // page size = 1 << page_shift
};

struct KvBatch {
    const int32_t* table;
    const int32_t* cu;
    const int32_t* len;
    int n_seq, max_pages;
};

// Rows of sequence b: [r0, r1), clamped into the call's T rows whatever cu
// holds, and the position of row r0.
struct SeqRows {
    int r0, r1, pos0;
};

__device__ __forceinline__ int cu_at(const KvBatch& bt, int b, int T) { return min(max(bt.cu[b], 0), T); }

__device__ __forceinline__ SeqRows seq_rows(const KvBatch& bt, int b, int T) {
    SeqRows s;
    s.r0 = cu_at(bt, b, T);
    s.r1 = max(cu_at(bt, b + 1, T), s.r0);
    s.pos0 = max(bt.len[b], 0) - (s.r1 - s.r0);   // negative: the first rows are before the sequence
    return s;
}

// Work units of a ragged batch without a prefix sum.  Sequence b has its
// units numbered from  first(b) = floor(cu[b] * mul / per) + extra * b,  and
// first(b + 1) - first(b) is at least the ceil(n_b * mul / per) + extra - 1
// units it can need, so a unit finds its sequence by bisection on cu alone.
// Numbers past a sequence's own units are empty.
__device__ __forceinline__ int unit_first(const KvBatch& bt, int b, int T, int mul, int per, int extra) {
    return (int)((int64_t)cu_at(bt, b, T) * mul / per) + extra * b;
}
__device__ __forceinline__ int unit_seq(const KvBatch& bt, int u, int T, int mul, int per, int extra) {
    int lo = 0, hi = bt.n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (unit_first(bt, mid, T, mul, per, extra) <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
inline int64_t unit_bound(int64_t n_seq, int64_t T, int64_t mul, int64_t per, int64_t extra) {
    return T * mul / per + extra * n_seq;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// two fp32 as packed bf16, round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const at_f32x2 x{a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, at_bf16x2));
}

hipError_t launch_kv_append(const KvCache& c, const KvBatch& bt, int D, const uint16_t* k, const uint16_t* v,
                            const uint16_t* q, int T, int Hq, const double* inv_freq, int rot, int interleaved,
                            uint16_t* q_out, hipStream_t st);

struct AttendArgs {
    KvCache c;
    KvBatch bt;
    const uint16_t* q;
    uint16_t* out;
    int T, Hq, G;            // G = Hq / Hkv query heads per key/value head
    float c2;                // scale * log2(e)
    int window, n_sink;
    const int32_t* list;     // selected: idx [T, cap]; packed: shared [groups, cap]
    const uint32_t* masks;   // packed
    const int32_t* lens;     // packed
    int cap, group;
    int splits;              // list kinds: key splits per unit
    int min_per;             // attend: least key tiles of a workgroup's range
    void* head;              // attend: the plan for the join
    float* part;             // partial rows and their statistics
};

// Launch of an attend call, fixed by its sizes alone so that the workspace
// size and the call agree.
struct AttendPlan {
    int mt;            // 16-row tiles per unit
    int64_t blocks;
    int splits;
    bool join;         // units may be cut: partial rows and a joining launch
    size_t head_bytes, ws_bytes;
};
AttendPlan attend_plan(int kind, int T, int Hq, int Hkv, int D, int n_seq, int64_t entries);

hipError_t launch_attend(int kind, int D, const AttendPlan& p, AttendArgs& a, void* ws, hipStream_t st);

}  // namespace ltk
