// int4_gemm.cu -- products of 16-bit rows with 4-bit weights, by groups of rows.
//
//   y[r] = row_scale[r] * x[src[r] / div] W[e]^T   for the rows r of group e
// with W[e][n][k] = (code - zero) * scale, scale and zero per row n and group of
// k.  code - zero is a small integer, exact in 16 bits, so a group's products
// are summed as they are and scaled once, in fp32.
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "int4.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

struct Int4Product {
    RaggedArgs r;          // N: weight rows per group
    const void* x;
    int64_t ldx, x_rows;
    const int32_t* src;    // [R] or null
    int32_t src_div;
    const uint32_t* codes; // [E, N, K / 8]
    const void* scales;    // [E, N, groups]
    const uint8_t* zeros;  // the same, or null
    int32_t groups, shift; // groups per weight row, log2 of their words
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// One warp per output column: its lanes take the words of the weight row in turn.
template <typename T, bool SWIGLU>
__global__ void __launch_bounds__(256) k_int4_product(const __grid_constant__ Int4Product p) {
    __shared__ RaggedTiles tiles;
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) ragged_tiles_build<32>(p.r, tiles, 1, lane);
    __syncthreads();
    const int e = blockIdx.y, n = blockIdx.x * 8 + warp, columns = SWIGLU ? p.r.N / 2 : p.r.N;
    if (n >= columns) return;
    const int words = p.r.K / 8;
    for (int row = tiles.lo[e]; row < tiles.hi[e]; ++row) {
        int64_t xr = row;
        bool have = true;
        if (p.src) {
            const int s = ld_dep(p.src + row);
            xr = s / p.src_div;
            have = s >= 0 && xr < p.x_rows;
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
            const int64_t w = static_cast<int64_t>(e) * p.r.N + (SWIGLU ? (n >> 7) * 256 + (n & 127) + 128 * h : n);
            for (int k = lane; have && k < words; k += 32) {
                const uint32_t q = ld_dep(p.codes + w * words + k);
                const int64_t g = w * p.groups + (k >> p.shift);
                const float s = to_float<T>(static_cast<const T*>(p.scales)[g]);
                const int zero = p.zeros ? p.zeros[g] : 8;
                const T* x = static_cast<const T*>(p.x) + xr * p.ldx + 8 * k;
                float part = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    part = fmaf(to_float<T>(x[i]), static_cast<float>(static_cast<int>(q >> (4 * (i >> 1) + 16 * (i & 1)) & 15u) - zero), part);
                sum[h] = fmaf(part, s, sum[h]);
            }
            sum[h] = warp_sum(sum[h]);
        }
        if (lane == 0) {
            float y = sum[0];
            if constexpr (SWIGLU) y = y / (1.0f + expf(-y)) * sum[1];
            if (p.r.row_scale) y *= ld_dep(p.r.row_scale + row);
            static_cast<T*>(p.r.out)[row * p.r.ldo + n] = from_float<T>(y);
        }
    }
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_grouped_gemm_int4(int32_t group, int32_t dtype, int64_t R, int32_t N, int32_t K, int32_t E,
                                              const void* x, int64_t x_rows, int64_t ldx, const int32_t* src,
                                              int32_t src_div, const void* w_codes, const void* w_scales,
                                              const void* w_zeros, const int32_t* offsets, const float* row_scale,
                                              int32_t swiglu, void* y, int64_t ldy, uint32_t* status, void* stream) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_last_error(MOE_ERR_INVALID_ARG, "dtype = %d is neither bf16 (0) nor f16 (1)", dtype);
    const moe_status_t s = static_cast<moe_status_t>(check_int4_row(group, K));
    if (s != MOE_OK) return s;
    if (R < 0 || N <= 0 || E <= 0)
        return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0, dimensions and groups > 0");
    if (N % (swiglu ? 128 : 8))
        return set_last_error(MOE_ERR_UNSUPPORTED, "N = %d is not a multiple of %d", N, swiglu ? 128 : 8);
    if (N > kRaggedMaxDim / 2) return set_last_error(MOE_ERR_UNSUPPORTED, "N = %d is more than 2^29", N);
    if (E > kRaggedMaxGroups) return set_last_error(MOE_ERR_UNSUPPORTED, "E = %d > 256", E);
    if (R > (1ll << 30)) return set_last_error(MOE_ERR_UNSUPPORTED, "too many rows for 32-bit row indices");
    if (R == 0) return MOE_OK;
    if (!x || !w_codes || !w_scales || (!offsets && E != 1) || !y)
        return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned(x, 16) || !aligned(w_codes, 16) || !aligned(y, 16) || !aligned(w_scales, 2))
        return set_last_error(MOE_ERR_INVALID_ARG, "x, w_codes and y must be 16-byte aligned, w_scales 2-byte");
    if (ldx < K || ldx % 8 || ldy < N || ldy % 8)
        return set_last_error(MOE_ERR_INVALID_ARG, "row strides must cover the row and be multiples of 8 elements");
    if (src ? (src_div <= 0 || x_rows <= 0) : x_rows < R)
        return set_last_error(MOE_ERR_INVALID_ARG, "x has too few rows, or src_div <= 0");
    Int4Product p{};
    p.r.offsets = offsets;
    p.r.R = static_cast<int32_t>(R);
    p.r.N = swiglu ? 2 * N : N;
    p.r.K = K;
    p.r.E = E;
    p.r.row_scale = row_scale;
    p.r.out = y;
    p.r.ldo = ldy;
    p.r.status = status;
    p.x = x;
    p.ldx = ldx;
    p.x_rows = x_rows;
    p.src = src;
    p.src_div = src_div;
    p.codes = static_cast<const uint32_t*>(w_codes);
    p.scales = w_scales;
    p.zeros = static_cast<const uint8_t*>(w_zeros);
    p.groups = (K + group - 1) / group;
    p.shift = group == 32 ? 2 : group == 64 ? 3 : 4;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid((N + 7) / 8, E);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, st, p); };
    const cudaError_t e = dtype == MOE_DTYPE_BF16
                              ? (swiglu ? go(k_int4_product<__nv_bfloat16, true>) : go(k_int4_product<__nv_bfloat16, false>))
                              : (swiglu ? go(k_int4_product<__half, true>) : go(k_int4_product<__half, false>));
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit weight product: %s", cudaGetErrorString(e));
}
