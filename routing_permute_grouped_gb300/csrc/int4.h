// int4.h -- what the 4-bit weights' quantiser and their two products share.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "ragged.cuh"

namespace moe {

// The rules on a row of codes; a moe_status_t.
int check_int4_row(int32_t group, int32_t K);

struct Int4Product {
    RaggedArgs r;          // N: weight rows per group
    const void* x;
    int64_t ldx;
    int32_t x_rows;
    int32_t columns;       // of y
    int32_t swiglu;
    const int32_t* src;    // [R] or null
    int32_t src_div;
    const uint8_t* codes;  // [E, N, K / 2]
    const void* scales;    // [E, N, groups]
    const uint8_t* zeros;  // the same, or null
    int32_t groups;        // per weight row
    int32_t whole;         // what a kernel reads of scales and zero points at once is aligned
    int32_t split;         // warps or CTAs that share a sum, a power of two
};

// The product with many token rows per group (int4_wide.cu)
template <typename T>
cudaError_t launch_int4_wide(int group, const Int4Product& p, cudaStream_t st);

#ifdef __CUDACC__
// Rows [lo, hi) of every group, its token tiles' width and its first work item
struct Int4Lists {
    int first[260], lo[260], hi[260], width[260];
};

struct Int4Item {
    int e, panel;
    int row, rows;  // token rows
};

// Thread e takes group e; all threads call, at least 256 of them.  Token tiles hold up
// to TILE rows and are as wide as one another, in steps of UNIT.  Where a group is
// bad, groups may overlap: each then starts past the ends of those before it.
template <int TILE, int UNIT>
__device__ __forceinline__ int int4_lists(const RaggedArgs& a, Int4Lists& s, int panels) {
    __shared__ int sums[8];
    const int e = threadIdx.x, lane = e & 31;
    bool bad = false;
    if (e < a.E) {
        const int2 g = group_rows(a, e, &bad);
        s.lo[e] = g.x;
        s.hi[e] = g.y;
    }
    if (__syncthreads_or(bad)) {
        if (e == 0)
            for (int i = 0, end = 0; i < a.E; ++i) {
                s.lo[i] = min(max(s.lo[i], end), s.hi[i]);
                end = max(end, s.hi[i]);
            }
        __syncthreads();
    }
    int n = 0;
    if (e < a.E) {
        const int len = s.hi[e] - s.lo[e], tiles = (len + TILE - 1) / TILE;
        s.width[e] = tiles ? ((len + tiles - 1) / tiles + UNIT - 1) / UNIT * UNIT : UNIT;
        n = tiles * panels;
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31 && e < 256) sums[e >> 5] = x;
    __syncthreads();
    int total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i == e >> 5) before = total;
        total += sums[i];
    }
    if (e < a.E) s.first[e] = before + x - n;
    if (e == 0) s.first[a.E] = total;
    __syncthreads();
    return total;
}

// Item t: its group by bisection; the token tiles of a panel follow one another,
// so that the CTAs that take them find its codes in L2.
__device__ __forceinline__ Int4Item int4_item(const Int4Lists& s, int n_groups, int panels, int t) {
    int e = 0, end = n_groups;  // first[e] <= t < first[end]
    while (end - e > 1) {
        const int mid = (e + end) >> 1;
        if (s.first[mid] <= t)
            e = mid;
        else
            end = mid;
    }
    Int4Item it;
    it.e = e;
    const unsigned i = t - s.first[e], tiles = static_cast<unsigned>(s.first[e + 1] - s.first[e]) / panels;
    const unsigned panel = i / tiles;
    const int width = s.width[e];
    it.panel = static_cast<int>(panel);
    it.row = s.lo[e] + static_cast<int>(i - panel * tiles) * width;
    it.rows = min(width, s.hi[e] - it.row);
    return it;
}

// The token row of row r of y; -1 where src picks none.
__device__ __forceinline__ int int4_token_row(const Int4Product& p, int r) {
    if (!p.src) return r;
    const int s = ld_dep(p.src + r), from = s / p.src_div;
    return s >= 0 && from < p.x_rows ? from : -1;
}

// Codes to 16-bit numbers.  Bits 0 .. 7 of a half word, with the rest zero, are the
// number bits * 2^-133 (bf16) or bits * 2^-24 (f16): below 2^-126 and 2^-14, and in the
// binade above, these types are linear.  So a masked nibble, in bits 0 .. 3 or 4 .. 7
// as it lies, is multiplied up and has its zero point subtracted in one operation,
// (code - zero) * 2^-6 or 2^-9 exactly, and two of a half word's four nibbles share a
// shift.  (Or-ing each shifted nibble into the mantissa of 128 and subtracting takes
// three shifts: 306 instead of 276 instructions for 32 x 128 weights.)
template <typename T>
struct Int4Wide;
template <>
struct Int4Wide<__nv_bfloat16> {
    using P = __nv_bfloat162;
    static constexpr uint32_t low = 0x7F007F00u, high = 0x7D007D00u;  // 2^127, 2^123
    static constexpr float unit = 0x1p-6f;
    static constexpr uint32_t format = 1;  // of tcgen05.mma's operands
};
template <>
struct Int4Wide<__half> {
    using P = __half2;
    static constexpr uint32_t low = 0x78007800u, high = 0x68006800u;  // 2^15, 2^11
    static constexpr float unit = 0x1p-9f;
    static constexpr uint32_t format = 0;
};
// Pair i of a word's eight codes, times Int4Wide<T>::unit; zero is -zero point in both
// halves in the same unit.
template <typename T>
__device__ __forceinline__ uint32_t int4_widen(uint32_t w, int i, uint32_t zero) {
    using P = typename Int4Wide<T>::P;
    const uint32_t bits = (i < 2 ? w : w >> 8) & (i & 1 ? 0x00F000F0u : 0x000F000Fu);
    const uint32_t up = i & 1 ? Int4Wide<T>::high : Int4Wide<T>::low;
    const P v = __hfma2(*reinterpret_cast<const P*>(&bits), *reinterpret_cast<const P*>(&up), *reinterpret_cast<const P*>(&zero));
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ uint32_t int4_zero(uint32_t point) {
    const float back = static_cast<float>(point) * -Int4Wide<T>::unit;
    return pack2(T(), back, back);
}
#endif

}  // namespace moe
