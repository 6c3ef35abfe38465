// ragged_gemm.cu -- matrix products grouped by expert on ragged row groups,
// bf16 or f16: y[r] = row_scale[r] * x[r] W[e]^T (or x[r] W[e]) and the weight
// gradient dW[e] = sum over e's rows of a[r]^T b[r].
//
// Plain tiles: a 16 x 16 thread block computes 64 x 64 outputs, operands
// staged through shared memory in steps of 16, fp32 accumulators.
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

template <typename T>
struct Strided {  // element (row, k) of a group's operand
    const T* p;
    int64_t row, k;
    __device__ float at(int64_t r, int64_t kk) const { return to_float(p[r * row + kk * k]); }
};

// The e-th group and 64-row tile of flat tile index t; e = -1 past the last.
__device__ int3 find_tile(const RaggedArgs& a, int t) {
    for (int e = 0; e < a.E; ++e) {
        const int2 g = group_rows(a, e);
        const int n = (g.y - g.x + 63) / 64;
        if (t < n) return make_int3(e, g.x + 64 * t, g.y);
        t -= n;
    }
    return make_int3(-1, 0, 0);
}

// 64 x 64 tile of A B^T: rows [m0, m1) of A, [n0, n1) of B, sum over [k0, k1)
template <typename T, typename Put>
__device__ void tile_product(const Strided<T>& A, int64_t m0, int64_t m1, const Strided<T>& B, int64_t n0,
                             int64_t n1, int64_t k0, int64_t k1, Put put) {
    __shared__ float sa[16][65], sb[16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k = k0; k < k1; k += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            const int kk = i & 15, r = i >> 4;
            sa[kk][r] = (m0 + r < m1 && k + kk < k1) ? A.at(m0 + r, k + kk) : 0.0f;
            sb[kk][r] = (n0 + r < n1 && k + kk < k1) ? B.at(n0 + r, k + kk) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[kk][ty + 16 * i] * sb[kk][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (m0 + ty + 16 * i < m1 && n0 + tx + 16 * j < n1) put(m0 + ty + 16 * i, n0 + tx + 16 * j, acc[i][j]);
}

template <typename T>
__global__ void __launch_bounds__(256) k_ragged_product(RaggedArgs a, const T* x, int64_t ldx, const T* w,
                                                        bool w_transposed) {
    pdl_trigger();
    pdl_wait();
    const int3 t = find_tile(a, blockIdx.y);
    if (t.x < 0) return;
    const Strided<T> X{x, ldx, 1};
    const Strided<T> W{w + static_cast<int64_t>(t.x) * a.N * a.K, w_transposed ? 1 : a.K, w_transposed ? a.N : 1};
    T* out = static_cast<T*>(a.out);
    tile_product(X, t.y, min(t.z, t.y + 64), W, static_cast<int64_t>(blockIdx.x) * 64, a.N, 0, a.K,
                 [&](int64_t r, int64_t n, float v) {
                     out[r * a.ldo + n] = from_float<T>(a.row_scale ? v * ld_dep(a.row_scale + r) : v);
                 });
}

template <typename T>
__global__ void __launch_bounds__(256) k_ragged_wgrad(RaggedArgs a, const T* x, int64_t ldx, const T* y, int64_t ldy) {
    pdl_trigger();
    pdl_wait();
    const int e = blockIdx.z;
    const int2 g = group_rows(a, e);
    const Strided<T> X{x, 1, ldx}, Y{y, 1, ldy};
    T* out = static_cast<T*>(a.out) + static_cast<int64_t>(e) * a.K * a.N;
    tile_product(X, static_cast<int64_t>(blockIdx.y) * 64, a.K, Y, static_cast<int64_t>(blockIdx.x) * 64, a.N, g.x,
                 g.y, [&](int64_t m, int64_t n, float v) { out[m * a.N + n] = from_float<T>(v); });
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status_t check_ragged(int32_t dtype, int64_t R, int32_t A, int32_t B, int32_t E) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_last_error(MOE_ERR_INVALID_ARG, "dtype = %d is neither bf16 (0) nor f16 (1)", dtype);
    if (R < 0 || A <= 0 || B <= 0 || E <= 0)
        return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0, dimensions and groups > 0");
    if (A % 8 || B % 8)
        return set_last_error(MOE_ERR_UNSUPPORTED, "dimensions %d and %d must be multiples of 8", A, B);
    if (E > kRaggedMaxGroups) return set_last_error(MOE_ERR_UNSUPPORTED, "E = %d > 256", E);
    if (R > (1ll << 30)) return set_last_error(MOE_ERR_UNSUPPORTED, "too many rows for 32-bit row indices");
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_grouped_gemm(int32_t dtype, int64_t R, int32_t N, int32_t K, int32_t E, const void* x,
                                         int64_t ldx, const void* w, int32_t w_transposed, const int32_t* offsets,
                                         const float* row_scale, void* y, int64_t ldy, uint32_t* status,
                                         void* stream) {
    const moe_status_t s = check_ragged(dtype, R, N, K, E);
    if (s != MOE_OK) return s;
    if (R == 0) return MOE_OK;
    if (!x || !w || !offsets || !y) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x) || !aligned16(w) || !aligned16(y))
        return set_last_error(MOE_ERR_INVALID_ARG, "x, w and y must be 16-byte aligned");
    if (ldx < K || ldx % 8 || ldy < N || ldy % 8)
        return set_last_error(MOE_ERR_INVALID_ARG,
                              "row strides must cover the row and be multiples of 8 elements");
    RaggedArgs a{};
    a.offsets = offsets;
    a.R = static_cast<int32_t>(R);
    a.N = N;
    a.K = K;
    a.E = E;
    a.row_scale = row_scale;
    a.out = y;
    a.ldo = ldy;
    a.status = status;
    const dim3 grid((N + 63) / 64, static_cast<unsigned>(R / 64 + E));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == MOE_DTYPE_BF16
                        ? launch_pdl(k_ragged_product<__nv_bfloat16>, grid, dim3(256), 0, st, a,
                                     static_cast<const __nv_bfloat16*>(x), ldx,
                                     static_cast<const __nv_bfloat16*>(w), w_transposed != 0)
                        : launch_pdl(k_ragged_product<__half>, grid, dim3(256), 0, st, a,
                                     static_cast<const __half*>(x), ldx, static_cast<const __half*>(w),
                                     w_transposed != 0);
    return e == cudaSuccess ? MOE_OK
                            : set_last_error(MOE_ERR_CUDA, "grouped product: %s", cudaGetErrorString(e));
}

extern "C" moe_status_t moe_grouped_wgrad(int32_t dtype, int64_t R, int32_t M, int32_t N, int32_t E, const void* a_,
                                          int64_t lda, const void* b, int64_t ldb, const int32_t* offsets, void* out,
                                          uint32_t* status, void* stream) {
    const moe_status_t s = check_ragged(dtype, R, M, N, E);
    if (s != MOE_OK) return s;
    if (!out || (R > 0 && (!a_ || !b || !offsets))) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(out) || (R > 0 && (!aligned16(a_) || !aligned16(b))))
        return set_last_error(MOE_ERR_INVALID_ARG, "a, b and out must be 16-byte aligned");
    if (R > 0 && (lda < M || lda % 8 || ldb < N || ldb % 8))
        return set_last_error(MOE_ERR_INVALID_ARG,
                              "row strides must cover the row and be multiples of 8 elements");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (R == 0) {
        e = cudaMemsetAsync(out, 0, static_cast<size_t>(E) * M * N * 2, st);
    } else {
        RaggedArgs a{};
        a.offsets = offsets;
        a.R = static_cast<int32_t>(R);
        a.N = N;
        a.K = M;
        a.E = E;
        a.out = out;
        a.status = status;
        const dim3 grid((N + 63) / 64, (M + 63) / 64, E);
        e = dtype == MOE_DTYPE_BF16
                ? launch_pdl(k_ragged_wgrad<__nv_bfloat16>, grid, dim3(256), 0, st, a,
                             static_cast<const __nv_bfloat16*>(a_), lda, static_cast<const __nv_bfloat16*>(b), ldb)
                : launch_pdl(k_ragged_wgrad<__half>, grid, dim3(256), 0, st, a, static_cast<const __half*>(a_), lda,
                             static_cast<const __half*>(b), ldb);
    }
    return e == cudaSuccess ? MOE_OK
                            : set_last_error(MOE_ERR_CUDA, "grouped weight gradient: %s", cudaGetErrorString(e));
}
