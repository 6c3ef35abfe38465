// fp4_gemm.cu -- the grouped product on 4-bit rows and weights with block
// scales: y[r] = row_scale[r] * gx * gw[e] * sum_k x[r, k] W[e][n, k].
//
// Plain tiles: a 16 x 16 thread block computes 64 x 64 outputs; both operands
// are widened to fp32 (exactly) into shared memory in steps of 32.
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

struct Fp4Rows {
    const uint8_t* codes;   // [rows, K / 2]
    const uint8_t* scales;  // [rows, stride]
};

template <bool NV>
__device__ void stage(float (&s)[32][65], const Fp4Rows& x, int64_t r0, int64_t r1, int k, int K, int stride) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
        const int r = i >> 4, b = i & 15;
        float2 v = make_float2(0.0f, 0.0f);
        if (r0 + r < r1) {
            const uint32_t code = ld_dep(x.scales + (r0 + r) * stride + (k + 2 * b) / (NV ? 16 : 32));
            const float sc = NV ? e4m3_to_f32(code) : e8m0_to_f32(code);
            v = e2m1x2_to_f32x2(ld_dep(x.codes + (r0 + r) * (K / 2) + k / 2 + b));
            v.x *= sc;
            v.y *= sc;
        }
        s[2 * b][r] = v.x;
        s[2 * b + 1][r] = v.y;
    }
}

template <bool NV>
__global__ void __launch_bounds__(256) k_ragged_product_fp4(RaggedArgs a, Fp4Rows x, Fp4Rows w, int stride) {
    __shared__ float sa[32][65], sb[32][65];
    pdl_trigger();
    pdl_wait();
    int t = blockIdx.y, e = 0, r0 = 0, r1 = 0;
    for (; e < a.E; ++e) {
        const int2 g = group_rows(a, e);
        const int n = (g.y - g.x + 63) / 64;
        if (t < n) {
            r0 = g.x + 64 * t;
            r1 = min(g.y, r0 + 64);
            break;
        }
        t -= n;
    }
    if (e == a.E) return;
    const int64_t n0 = static_cast<int64_t>(e) * a.N + blockIdx.x * 64;
    const int64_t n1 = static_cast<int64_t>(e + 1) * a.N;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k = 0; k < a.K; k += 32) {
        stage<NV>(sa, x, r0, r1, k, a.K, stride);
        stage<NV>(sb, w, n0, n1, k, a.K, stride);
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 32; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[kk][ty + 16 * i] * sb[kk][tx + 16 * j];
        __syncthreads();
    }
    const float g = (a.x_scale ? ld_dep(a.x_scale) : 1.0f) * (a.w_scale ? ld_dep(a.w_scale + e) : 1.0f);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (r < r1 && n < n1)
                out[r * a.ldo + n - static_cast<int64_t>(e) * a.N] =
                    __float2bfloat16_rn(acc[i][j] * g * (a.row_scale ? ld_dep(a.row_scale + r) : 1.0f));
        }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_grouped_gemm_fp4(int32_t fmt, int64_t R, int32_t N, int32_t K, int32_t E, const void* x_codes,
                                             const void* x_scales, const void* w_codes, const void* w_scales,
                                             const int32_t* offsets, const float* x_scale, const float* w_scale,
                                             const float* row_scale, void* y, int64_t ldy, uint32_t* status,
                                             void* stream) {
    if (fmt != MOE_FP4_MX && fmt != MOE_FP4_NV)
        return set_last_error(MOE_ERR_INVALID_ARG, "format = %d is neither MX (0) nor NV (1)", fmt);
    if (R < 0 || N <= 0 || K <= 0 || E <= 0)
        return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0, dimensions and groups > 0");
    if (K % 32 || N % 8)
        return set_last_error(MOE_ERR_UNSUPPORTED, "K = %d must be a multiple of 32 and N = %d of 8", K, N);
    if (E > kRaggedMaxGroups) return set_last_error(MOE_ERR_UNSUPPORTED, "E = %d > 256", E);
    if (R > (1ll << 30)) return set_last_error(MOE_ERR_UNSUPPORTED, "too many rows for 32-bit row indices");
    if (R == 0) return MOE_OK;
    if (!x_codes || !x_scales || !w_codes || !w_scales || !offsets || !y)
        return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y))
        return set_last_error(MOE_ERR_INVALID_ARG, "codes, scales and y must be 16-byte aligned");
    if (ldy < N || ldy % 8)
        return set_last_error(MOE_ERR_INVALID_ARG, "the row stride must cover the row and be a multiple of 8 elements");
    RaggedArgs a{};
    a.offsets = offsets;
    a.R = static_cast<int32_t>(R);
    a.N = N;
    a.K = K;
    a.E = E;
    a.row_scale = row_scale;
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.out = y;
    a.ldo = ldy;
    a.status = status;
    const Fp4Rows x{static_cast<const uint8_t*>(x_codes), static_cast<const uint8_t*>(x_scales)};
    const Fp4Rows w{static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales)};
    const int stride = static_cast<int>(moe_fp4_scale_stride(fmt, K));
    const dim3 grid((N + 63) / 64, static_cast<unsigned>(R / 64 + E));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = fmt == MOE_FP4_NV ? launch_pdl(k_ragged_product_fp4<true>, grid, dim3(256), 0, st, a, x, w, stride)
                                      : launch_pdl(k_ragged_product_fp4<false>, grid, dim3(256), 0, st, a, x, w, stride);
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit grouped product: %s", cudaGetErrorString(e));
}
