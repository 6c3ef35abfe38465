// fp4.cu -- rows to and from 4-bit codes with block scales.
//
// A block of consecutive elements of a row shares one scale byte and holds
// e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte,
// the even element in the low nibble:
//   MX  32 elements, scale 2^(byte - 127), the smallest power of two with
//       amax <= 6 * scale (no element saturates)
//   NV  16 elements, scale e4m3(min(448, amax / (6 g))) * g, g the tensor's
//       fp32 scale
// code = the e2m1 value nearest to x / scale, ties to even.  Every step is an
// fp32 operation with one rounding (the power-of-two steps have none), so the
// codes are fixed by the inputs alone.
//
// One thread quantises one block; amax is taken on the bit patterns, where
// NaN and infinity order above every number, and marks the block's scale NaN.
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

struct QuantArgs {
    const void* x;
    int64_t ldx;
    int64_t rows;        // output rows
    int64_t x_rows;      // rows of x
    const int32_t* src;  // [rows] or null
    int32_t src_div;
    int32_t K;           // output columns
    int32_t stride;      // scale bytes per row
    const float* tensor_scale;
    uint8_t* codes;
    uint8_t* scales;
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

template <typename T, int N>
__device__ __forceinline__ void load_values(const T* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        const uint4 u = __ldcg(reinterpret_cast<const uint4*>(p + i));
        const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i + j] = to_float(t[j]);
    }
}

template <typename T, bool NV, bool SWIGLU>
__global__ void __launch_bounds__(256) k_quantize_fp4(const QuantArgs a) {
    constexpr int B = NV ? 16 : 32;
    pdl_trigger();
    pdl_wait();
    const int64_t total = a.rows * a.stride;
    const int nb = a.K / B;
    const float g = NV && a.tensor_scale ? ld_dep(a.tensor_scale) : 1.0f;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / a.stride;
        const int b = static_cast<int>(i - r * a.stride);
        if (b >= nb) {  // the padding of a scale row
            a.scales[i] = 0;
            continue;
        }
        int64_t xr = r;
        bool have = true;
        if (a.src) {
            const int s = ld_dep(a.src + r);
            xr = s / a.src_div;
            have = s >= 0 && xr < a.x_rows;
        }
        float v[B];
#pragma unroll
        for (int j = 0; j < B; ++j) v[j] = 0.0f;
        if (have) {
            const T* row = static_cast<const T*>(a.x) + xr * a.ldx;
            if constexpr (SWIGLU) {  // gate and up columns interleaved per 128
                const int c = b * B;
                float u[B];
                const T* p = row + (c >> 7) * 256 + (c & 127);
                load_values<T, B>(p, v);
                load_values<T, B>(p + 128, u);
#pragma unroll
                for (int j = 0; j < B; ++j) v[j] = to_float(from_float<T>(silu(v[j]) * u[j]));
            } else {
                load_values<T, B>(row + static_cast<int64_t>(b) * B, v);
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < B; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        uint32_t code;
        uint32_t q[B / 8];
        if (top >= 0x7F800000u) {  // a NaN or infinity: the whole block is NaN
            code = NV ? 0x7Fu : 0xFFu;
#pragma unroll
            for (int j = 0; j < B / 8; ++j) q[j] = 0;
        } else if constexpr (NV) {
            code = f32_to_e4m3(fminf(__uint_as_float(top) / (g * 6.0f), 448.0f));
            const float s = e4m3_to_f32(code) * g;
#pragma unroll
            for (int j = 0; j < B / 8; ++j) {
                q[j] = 0;
                if (s > 0.0f)
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        q[j] |= f32x2_to_e2m1x2(v[8 * j + 2 * p] / s, v[8 * j + 2 * p + 1] / s) << (8 * p);
            }
        } else {
            // amax = 1.m * 2^(e - 127) <= 1.5 * 2^2 * 2^(code - 127)
            const int e = static_cast<int>(top >> 23);
            const int c = e - ((top & 0x7FFFFFu) <= 0x400000u ? 2 : 1);
            code = top ? static_cast<uint32_t>(max(c, 0)) : 127u;
            const float inv = __uint_as_float((254u - code) << 23);  // 2^(127 - code)
#pragma unroll
            for (int j = 0; j < B / 8; ++j) {
                q[j] = 0;
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    q[j] |= f32x2_to_e2m1x2(v[8 * j + 2 * p] * inv, v[8 * j + 2 * p + 1] * inv) << (8 * p);
            }
        }
        a.scales[i] = static_cast<uint8_t>(code);
        uint8_t* out = a.codes + r * (a.K / 2) + static_cast<int64_t>(b) * (B / 2);
        if constexpr (NV)
            *reinterpret_cast<uint2*>(out) = make_uint2(q[0], q[1]);
        else
            *reinterpret_cast<uint4*>(out) = make_uint4(q[0], q[1], q[2], q[3]);
    }
}

// Sixteen elements per thread: value = e2m1 * scale (* g), one rounding each
template <typename T, bool NV>
__global__ void __launch_bounds__(256)
    k_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, int stride,
                     const float* tensor_scale, T* out, int64_t ldo) {
    pdl_trigger();
    pdl_wait();
    const int per = K / 16;
    const int64_t total = rows * per;
    const float g = NV && tensor_scale ? ld_dep(tensor_scale) : 1.0f;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / per;
        const int c = static_cast<int>(i - r * per) * 16;
        const uint2 q = __ldcg(reinterpret_cast<const uint2*>(codes + r * (K / 2) + c / 2));
        const uint32_t code = ld_dep(scales + r * stride + c / (NV ? 16 : 32));
        const float s = NV ? e4m3_to_f32(code) : e8m0_to_f32(code);
        T v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = e2m1x2_to_f32x2(((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 0xFFu);
            v[2 * j] = from_float<T>(f.x * s * g);
            v[2 * j + 1] = from_float<T>(f.y * s * g);
        }
        uint4* o = reinterpret_cast<uint4*>(out + r * ldo + c);
        o[0] = reinterpret_cast<const uint4*>(v)[0];
        o[1] = reinterpret_cast<const uint4*>(v)[1];
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status_t check_fp4(int32_t fmt, int64_t rows, int32_t K) {
    if (fmt != MOE_FP4_MX && fmt != MOE_FP4_NV)
        return set_last_error(MOE_ERR_INVALID_ARG, "format = %d is neither MX (0) nor NV (1)", fmt);
    if (rows < 0 || K <= 0) return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0 and K > 0");
    if (K % 32) return set_last_error(MOE_ERR_UNSUPPORTED, "K = %d is not a multiple of 32", K);
    if (rows > (1ll << 40) / K) return set_last_error(MOE_ERR_UNSUPPORTED, "tensor too large");
    return MOE_OK;
}

unsigned blocks_for(int64_t threads) {
    const int64_t b = (threads + 255) / 256;
    const int64_t most = static_cast<int64_t>(num_sms()) * 64;
    return static_cast<unsigned>(b < most ? b : most);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_fp4_scale_stride(int32_t fmt, int32_t K) {
    if ((fmt != MOE_FP4_MX && fmt != MOE_FP4_NV) || K <= 0 || K % 32) return 0;
    const size_t n = static_cast<size_t>(K) / (fmt == MOE_FP4_MX ? 32 : 16);
    return (n + 15) / 16 * 16;
}

extern "C" moe_status_t moe_quantize_fp4(int32_t fmt, int32_t dtype, int64_t rows, int32_t K, const void* x,
                                         int64_t x_rows, int64_t ldx, const int32_t* src, int32_t src_div,
                                         int32_t swiglu, const float* tensor_scale, void* codes, void* scales,
                                         void* stream) {
    const moe_status_t s = check_fp4(fmt, rows, K);
    if (s != MOE_OK) return s;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_last_error(MOE_ERR_INVALID_ARG, "dtype = %d is neither bf16 (0) nor f16 (1)", dtype);
    if (swiglu && K % 128)
        return set_last_error(MOE_ERR_UNSUPPORTED, "SwiGLU input is interleaved per 128 columns: K = %d is not a multiple",
                              K);
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales))
        return set_last_error(MOE_ERR_INVALID_ARG, "x, codes and scales must be 16-byte aligned");
    const int64_t cols = swiglu ? 2 * static_cast<int64_t>(K) : K;
    if (ldx < cols || ldx % 8)
        return set_last_error(MOE_ERR_INVALID_ARG, "the row stride must cover the row and be a multiple of 8 elements");
    if (src ? (src_div <= 0 || x_rows <= 0) : x_rows < rows)
        return set_last_error(MOE_ERR_INVALID_ARG, "x has too few rows, or src_div <= 0");
    QuantArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.rows = rows;
    a.x_rows = x_rows;
    a.src = src;
    a.src_div = src_div;
    a.K = K;
    a.stride = static_cast<int32_t>(moe_fp4_scale_stride(fmt, K));
    a.tensor_scale = tensor_scale;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales);
    const dim3 grid(blocks_for(rows * a.stride));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool nv = fmt == MOE_FP4_NV, bf = dtype == MOE_DTYPE_BF16;
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, st, a); };
    cudaError_t e;
    if (bf)
        e = nv ? (swiglu ? go(k_quantize_fp4<__nv_bfloat16, true, true>) : go(k_quantize_fp4<__nv_bfloat16, true, false>))
               : (swiglu ? go(k_quantize_fp4<__nv_bfloat16, false, true>)
                         : go(k_quantize_fp4<__nv_bfloat16, false, false>));
    else
        e = nv ? (swiglu ? go(k_quantize_fp4<__half, true, true>) : go(k_quantize_fp4<__half, true, false>))
               : (swiglu ? go(k_quantize_fp4<__half, false, true>) : go(k_quantize_fp4<__half, false, false>));
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit quantisation: %s", cudaGetErrorString(e));
}

extern "C" moe_status_t moe_dequantize_fp4(int32_t fmt, int32_t dtype, int64_t rows, int32_t K, const void* codes,
                                           const void* scales, const float* tensor_scale, void* out, int64_t ldo,
                                           void* stream) {
    const moe_status_t s = check_fp4(fmt, rows, K);
    if (s != MOE_OK) return s;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_last_error(MOE_ERR_INVALID_ARG, "dtype = %d is neither bf16 (0) nor f16 (1)", dtype);
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !out) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(out))
        return set_last_error(MOE_ERR_INVALID_ARG, "codes, scales and out must be 16-byte aligned");
    if (ldo < K || ldo % 8)
        return set_last_error(MOE_ERR_INVALID_ARG, "the row stride must cover the row and be a multiple of 8 elements");
    const int stride = static_cast<int>(moe_fp4_scale_stride(fmt, K));
    const dim3 grid(blocks_for(rows * (K / 16)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel, auto* o) {
        return launch_pdl(kernel, grid, dim3(256), 0, st, static_cast<const uint8_t*>(codes),
                          static_cast<const uint8_t*>(scales), rows, K, stride, tensor_scale, o, ldo);
    };
    const bool nv = fmt == MOE_FP4_NV;
    cudaError_t e;
    if (dtype == MOE_DTYPE_BF16) {
        auto* o = static_cast<__nv_bfloat16*>(out);
        e = nv ? go(k_dequantize_fp4<__nv_bfloat16, true>, o) : go(k_dequantize_fp4<__nv_bfloat16, false>, o);
    } else {
        auto* o = static_cast<__half*>(out);
        e = nv ? go(k_dequantize_fp4<__half, true>, o) : go(k_dequantize_fp4<__half, false>, o);
    }
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit values: %s", cudaGetErrorString(e));
}
