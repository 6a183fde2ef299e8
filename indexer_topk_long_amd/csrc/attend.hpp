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
// Both searches try the sequence that an even batch would give first (one
// round of loads instead of log2(n_seq) dependent ones) and its neighbours.
__device__ __forceinline__ int unit_seq(const KvBatch& bt, int u, int T, int mul, int per, int extra) {
    const int last = bt.n_seq - 1;
    if (last <= 0) return 0;
    const int64_t all = (int64_t)T * mul / per + (int64_t)extra * bt.n_seq;
    const int g = min((int)((int64_t)u * bt.n_seq / max(all, (int64_t)1)), last);
    const int f0 = unit_first(bt, max(g - 1, 0), T, mul, per, extra), f1 = unit_first(bt, g, T, mul, per, extra);
    const int f2 = unit_first(bt, min(g + 1, last), T, mul, per, extra);
    const int f3 = unit_first(bt, min(g + 2, last), T, mul, per, extra);
    if (g > 0 && f0 <= u && u < f1) return g - 1;
    if (f1 <= u && (g == last || u < f2)) return g;
    if (g < last && f2 <= u && (g + 1 == last || u < f3)) return g + 1;
    int lo = 0, hi = last;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (unit_first(bt, mid, T, mul, per, extra) <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
// The sequence of a row: the last one that begins at or before it (so not an
// empty one, where the row is in any).
__device__ __forceinline__ int row_seq(const KvBatch& bt, int row, int T) {
    const int last = bt.n_seq - 1;
    if (last <= 0) return 0;
    const int g = min((int)((int64_t)row * bt.n_seq / max(T, 1)), last);
    if (cu_at(bt, g, T) <= row && row < cu_at(bt, g + 1, T)) return g;
    int lo = 0, hi = last;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu_at(bt, mid, T) <= row)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
inline int64_t unit_bound(int64_t n_seq, int64_t T, int64_t mul, int64_t per, int64_t extra) {
    return T * mul / per + extra * n_seq;
}

// A value that all lanes hold, in scalar registers: what is derived from it
// (page ids above all) is then loaded through the scalar cache and does not
// queue behind the tiles' loads.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32) | (uint32_t)uniform((int)x));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// two fp32 as packed bf16, round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const at_f32x2 x{a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, at_bf16x2));
}

// Running softmax of a row: weights are 2^(y - m).  The reference m moves only
// when a score passes it by more than kSlack (weights up to 256 in fp16), or
// at the row's first visible key: until then m is 0 and `over`, the excess
// that moves it, is -infinity.
constexpr float kSlack = 8.0f;
constexpr float kNoRef = -1e30f;     // reference of a part that saw no key

// 8 e4m3 bytes as bf16, exact
__device__ __forceinline__ at_bf16x8 bf16_of(uint32_t a, uint32_t b) {
    const at_bf16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const at_bf16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const at_bf16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const at_bf16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return at_bf16x8{x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
}

// Keys whose value scale is below this have their share of the divisor formed
// by an exponential of its own, 2^((y - m) - log2(vs)), and not as 2^(y - m)
// times 1 / vs: beside a value scale of up to 2^64, a weight that matters to the
// divisor can lie below fp32's range (2^-126) in the first form.  A key at or
// above it whose weight falls below that range is at most 2^-38 of the divisor.
constexpr float kSmallScale = 0x1p-24f;

// Constants of a key: scale log2(e) ks, log2(vs), 1 / vs (0 for a small scale).
// Dense tiles have one set per half (a page holds at least 16 keys), listed keys
// one each.
struct PageScale {
    float c_, lv_, iv_;
    __device__ __forceinline__ float c(int) const { return c_; }
    __device__ __forceinline__ float lv(int) const { return lv_; }
    __device__ __forceinline__ float iv(int) const { return iv_; }
};
// v_log_f32 is base 2; both it and v_rcp_f32 are exact on powers of two and
// within 1 ulp elsewhere.
__device__ __forceinline__ PageScale page_scale(float c2, float ks, float vs) {
    return PageScale{c2 * ks, __builtin_amdgcn_logf(vs), vs >= kSmallScale ? __builtin_amdgcn_rcpf(vs) : 0.0f};
}
__device__ __forceinline__ bool is_small(const PageScale& s) { return __float_as_uint(s.iv_) == 0u; }
// The divisor's share of a key of a small scale, for y relative to the row's reference.
__device__ __forceinline__ float small_share(float y, float lv, float iv) {
    return iv == 0.0f ? __builtin_amdgcn_exp2f(y - lv) : 0.0f;
}
// 2^d as the square of h = 2^(d / 2).  A divisor is scaled by h twice: d can pass
// the range of one factor (value scales 2^128 apart) where the product is one
// that counts.
struct Factor {
    float h, f;
    explicit __device__ __forceinline__ Factor(float d) : h(__builtin_amdgcn_exp2f(0.5f * d)), f(h * h) {}
    __device__ __forceinline__ float divisor(float x) const { return x * h * h; }
};

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
    void* head;              // attend: what the join needs to know
    float* part;             // partial rows and their statistics
    // sequences that share their first tokens: group j is the sequences groups[j] .. groups[j + 1] - 1
    const int32_t* groups;
    const int32_t* shared_len;
    int n_group;
    int32_t* own;            // [n_seq]: keys that a sequence does not see for itself, as the shared keys' launch notes them
    float* prior;            // [T * Hq][D + kPriorTail]: every row's sums over its group's shared keys
};

// What a launch of the dense kernels attends to: all keys of a sequence; the
// keys that a group shares, met by the rows of all its sequences and left as
// sums in `prior`; or a sequence's own keys behind those, beginning from them.
// (64 rows, 64 heads on 8, D = 128: 32,768 shared tokens take 96 to 99 us in the wide
// kernel, 700 to 720 TFLOP/s, and 8 to join; up to 1,000 own tokens each 23 and 5.
// 64 sequences of eight rows each: 580 us in all with 100 own tokens, 611 with 1,000.)
enum Part { kAllKeys, kSharedKeys, kOwnKeys };
// A row of prior: D sums, the reference m, the divisor l.
constexpr int kPriorTail = 4;

__device__ __forceinline__ int group_at(const AttendArgs& a, int j) { return min(max(a.groups[j], 0), a.bt.n_seq); }
__device__ __forceinline__ int shared_keys(const AttendArgs& a, int j) {
    return min(max(a.shared_len[j], 0), a.bt.max_pages << a.c.page_shift);
}
// Keys that sequence b does not see for itself: those its group shares.  Found
// once, by the shared keys' launch (its threads all call note_own): looked for by
// every workgroup of the second launch, several times a unit, it cost the
// smallest calls 7 us.
__device__ __forceinline__ int own_from(const AttendArgs& a, int b) { return a.own[b]; }
__device__ __forceinline__ int find_own(const AttendArgs& a, int b) {
    int lo = 0, hi = a.n_group - 1;
    if (hi < 0) return 0;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (group_at(a, mid) <= b)
            lo = mid;
        else
            hi = mid - 1;
    }
    return group_at(a, lo) <= b && b < group_at(a, lo + 1) ? shared_keys(a, lo) : 0;
}
__device__ __forceinline__ void note_own(const AttendArgs& a) {
    const int64_t threads = (int64_t)gridDim.x * blockDim.x;
    for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < a.bt.n_seq; b += threads)
        a.own[b] = find_own(a, (int)b);
}
// The entries of the batch as a launch sees it: sequences, or groups with the
// rows of all their sequences.
template <int PART>
__device__ __forceinline__ int batch_size(const AttendArgs& a) {
    return PART == kSharedKeys ? a.n_group : a.bt.n_seq;
}
template <int PART>
__device__ __forceinline__ SeqRows batch_rows(const AttendArgs& a, int b) {
    if constexpr (PART == kSharedKeys) {
        SeqRows s;
        s.r0 = cu_at(a.bt, group_at(a, b), a.T);
        s.r1 = max(cu_at(a.bt, group_at(a, b + 1), a.T), s.r0);
        s.pos0 = 0;   // (rows see the shared keys whatever their positions are)
        return s;
    } else {
        return seq_rows(a.bt, b, a.T);
    }
}
template <int PART>
__device__ __forceinline__ const int32_t* batch_table(const AttendArgs& a, int b) {
    const int row = PART == kSharedKeys ? min(group_at(a, b), a.bt.n_seq - 1) : b;
    return a.bt.table + (size_t)row * a.bt.max_pages;
}

// Page ids and scales of the next 64 groups of 16 keys, one a lane, so that a
// loop over keys reads the page table and the scales once per 64 groups, a
// block ahead, and takes each step's from a lane.  (Loaded through the scalar
// cache step by step, every wait for LDS or for a scale would also wait for
// the ids of the step after, since scalar loads return out of order.)
struct PageLanes {
    int id, ahead;      // checked ids of this block (-1: no page, or no key of it is seen); the next block's as read
    float ks, vs;       // as read
    PageScale s;
    uint64_t small;     // lanes whose group's value scale is small

    // key_of(block): first key of the lane's group, < 0 past the end.
    template <class KeyOf>
    __device__ __forceinline__ void read(const int32_t* table, const AttendArgs& a, int block, KeyOf key_of) {
        const int key = key_of(block);
        ahead = key >= 0 ? table[min(key >> a.c.page_shift, a.bt.max_pages - 1)] : -1;
    }
    // Makes `block` the current one; its scales are on their way afterwards.
    template <class KeyOf, class Seen>
    __device__ __forceinline__ void turn(const int32_t* table, const AttendArgs& a, int h, int block, KeyOf key_of,
                                         Seen seen) {
        const int key = key_of(block);
        id = (key >= 0) & (ahead >= 0) & (ahead < a.c.n_pages) & seen(key) ? ahead : -1;
        read(table, a, block + 1, key_of);
        const size_t tile = (size_t)max(id, 0) * a.c.Hkv + h;
        ks = 1.0f, vs = 1.0f;
        if (id >= 0) ks = a.c.ks[tile], vs = a.c.vs[tile];
    }
    __device__ __forceinline__ void scales(float c2) {
        s = page_scale(c2, ks, vs);
        small = __ballot(is_small(s));
    }
    __device__ __forceinline__ uint32_t any_small(int lane, int groups) const {
        return (uint32_t)(small >> lane) & ((1u << groups) - 1u);
    }
    __device__ __forceinline__ int page(int lane) const { return __builtin_amdgcn_readlane(id, lane); }
    __device__ __forceinline__ PageScale scale(int lane) const {
        return PageScale{lane_of(s.c_, lane), lane_of(s.lv_, lane), lane_of(s.iv_, lane)};
    }
    static __device__ __forceinline__ float lane_of(float x, int lane) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
    }
};

// A launch has fewer than 2^32 threads.
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= (int64_t)0xffffffff / threads; }

// Launch of an append, fixed by its sizes.
struct AppendPlan {
    int vec, heads_per, units;
    int64_t blocks;
    bool fits;
};
AppendPlan append_plan(int T, int Hq, int Hkv, int D, int n_seq, int page, int rot, bool queries);
hipError_t launch_kv_append(const AppendPlan& p, const KvCache& c, const KvBatch& bt, int D, const uint16_t* k,
                            const uint16_t* v, const uint16_t* q, int T, int Hq, const double* inv_freq, int rot,
                            int interleaved, uint16_t* q_out, hipStream_t st);

bool kv_read_fits(int T, int D);
hipError_t launch_kv_read(const KvCache& c, const KvBatch& bt, int T, int D, int type, void* k, void* v, hipStream_t st);

// Launch of an attend call, fixed by its sizes alone so that the workspace
// size and the call agree.
struct AttendPlan {
    bool tile;         // the kernels of attend_tile.hip, else those of attend.hip
    int mt;            // attend.hip: 16-row tiles per unit
    int waves;         // attend_tile.hip: 32 rows each
    int64_t blocks;
    int splits;
    bool join;         // units may be cut: partial rows and a joining launch
    size_t head_bytes, ws_bytes;
    bool fits() const { return grid_fits(blocks, tile ? 64 * waves : 256); }
};
// `group` is the packed kind's (else 0).
AttendPlan attend_plan(int kind, int T, int Hq, int Hkv, int D, int n_seq, int64_t entries, int group);
// A bound of ws_bytes over all calls of no more rows, sequences and entries.
size_t attend_workspace_bound(int kind, int T, int Hq, int Hkv, int D, int n_seq, int64_t entries, int group);
// Units past this many change no launch: each is a range of keys at least.
constexpr int64_t kManyUnits = 1 << 20;
// attend_tile.hip: units of 32 `waves` rows; `units` bounds their number.
AttendPlan attend_tile_plan(int waves, int64_t units, int D, int64_t entries);
AttendPlan attend_tile_list_plan(int64_t groups, int64_t pairs, int Hkv, int D, int64_t entries);
bool attend_tile_wide(int64_t rows, int n_seq, int64_t work);

hipError_t launch_attend(int kind, int D, const AttendPlan& p, AttendArgs& a, void* ws, hipStream_t st, int part = kAllKeys);
hipError_t launch_attend_tile(int kind, int D, const AttendPlan& p, const AttendArgs& a, hipStream_t st, int part = kAllKeys);

}  // namespace ltk
