// kv_read.hip -- rows of the paged e4m3 cache back in 16 or 32 bits: bound by
// the bytes, one read and two (or four) written per value.
//
// A thread takes 8 bytes of a row and head, keys and values alike, and the
// same of the heads after it: the row's sequence, position and page are looked
// up once for all of them.  82,870 rows of eight heads (D = 128, to bf16) take 102 to
// 104 us, 4.9 TB/s, where a large copy reaches 5.05; 100 rows 2.9 us.
#include <algorithm>

#include "prompt.hpp"

namespace ltk {

namespace {

struct ReadArgs {
    KvCache c;
    KvBatch bt;
    int T;
    void *k, *v;
};

constexpr int kThreads = 256;

// The values of 8 bytes.  (16 bytes a thread, and so two stores 32 bytes apart
// between lanes: 82,870 rows of eight heads, D = 128, to bf16: 117 us against 104, 4.9 TB/s;
// stores past the caches: 182.)
template <int TYPE>
__device__ __forceinline__ void store8(void* out, int64_t at, const at_u32x2& w, float scale) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const at_f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        x[4 * i] = lo[0] * scale, x[4 * i + 1] = lo[1] * scale;
        x[4 * i + 2] = hi[0] * scale, x[4 * i + 3] = hi[1] * scale;
    }
    if constexpr (TYPE == LTK_ROWS_FP32) {
        float* p = static_cast<float*>(out) + at;
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<at_f32x4*>(p + 4 * i) = at_f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    } else {
        using E = std::conditional_t<TYPE == LTK_ROWS_BF16, PrBf16, PrF16>;
        *reinterpret_cast<at_u32x4*>(static_cast<uint16_t*>(out) + at) =
            at_u32x4{E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]), E::pack(x[6], x[7])};
    }
}

template <int TYPE, int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(ReadArgs a) {
    constexpr int L = D / 8;   // threads of a row
    const int64_t row = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const int d = 8 * (threadIdx.x % L);
    if (row >= a.T) return;
    const int t = (int)row, b = row_seq(a.bt, t, a.T);
    // T may end inside a sequence: its rows keep their positions, which count from its last one
    const int r1 = a.bt.cu[b + 1];
    if (t < a.bt.cu[b] || t >= r1) return;
    const int64_t pos = (int64_t)max(a.bt.len[b], 0) - r1 + t, page = pos >> a.c.page_shift;
    int id = -1;
    if (pos >= 0 && page < a.bt.max_pages) id = a.bt.table[(size_t)b * a.bt.max_pages + page];
    const bool have = id >= 0 && id < a.c.n_pages;
    const int slot = (int)pos & ((1 << a.c.page_shift) - 1);
#pragma unroll 4
    for (int h = blockIdx.y; h < a.c.Hkv; h += gridDim.y) {
        at_u32x2 kw{0u, 0u}, vw = kw;
        float ks = 0.0f, vs = 0.0f;
        if (have) {
            const size_t pg = (size_t)id * a.c.Hkv + h, at = ((pg << a.c.page_shift) + slot) * D + d;
            kw = *reinterpret_cast<const at_u32x2*>(a.c.k + at);
            vw = *reinterpret_cast<const at_u32x2*>(a.c.v + at);
            ks = a.c.ks[pg];
            vs = a.c.vs[pg];
        }
        const int64_t at = (row * a.c.Hkv + h) * D + d;
        store8<TYPE>(a.k, at, kw, ks);
        store8<TYPE>(a.v, at, vw, vs);
    }
}

template <int TYPE>
hipError_t launch(const ReadArgs& a, int D, const dim3& grid, hipStream_t st) {
    if (D == 64)
        kv_read_kernel<TYPE, 64><<<grid, kThreads, 0, st>>>(a);
    else
        kv_read_kernel<TYPE, 128><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

static int64_t row_blocks(int T, int D) { return ((int64_t)T * (D / 8) + kThreads - 1) / kThreads; }

bool kv_read_fits(int T, int D) { return grid_fits(row_blocks(T, D), kThreads); }

hipError_t launch_kv_read(const KvCache& c, const KvBatch& bt, int T, int D, int type, void* k, void* v, hipStream_t st) {
    const int64_t blocks = row_blocks(T, D);
    const int64_t spread = std::max<int64_t>(1, std::min<int64_t>(c.Hkv, 2048 / blocks));
    const ReadArgs a{c, bt, T, k, v};
    const dim3 grid((unsigned)blocks, (unsigned)spread);
    if (type == LTK_ROWS_BF16) return launch<LTK_ROWS_BF16>(a, D, grid, st);
    if (type == LTK_ROWS_FP16) return launch<LTK_ROWS_FP16>(a, D, grid, st);
    return launch<LTK_ROWS_FP32>(a, D, grid, st);
}

}  // namespace ltk
