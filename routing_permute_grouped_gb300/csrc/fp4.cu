// fp4.cu -- rows to and from 4-bit codes with block scales.
//
// A block of consecutive elements of a row shares one scale byte and holds
// e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte,
// the even element in the low nibble:
//   MX  32 elements, scale 2^(byte - 127), the smallest power of two with
//       amax <= 6 * scale (no element saturates; the conversion that OCP's text
//       gives takes 2^(floor(log2 amax) - 2) and lets the top of a block saturate,
//       half this scale where amax's significand is above 1.5)
//   NV  16 elements, scale e4m3(min(448, amax / (6 g))) * g, g the tensor's
//       fp32 scale
// code = the e2m1 value nearest to x / scale, ties to even.  Every step is an
// fp32 operation with one rounding (the power-of-two steps have none), so the
// codes are fixed by the inputs alone.
//
// Dequantising is bound by memory: a thread takes 8 elements (4 bytes of codes,
// 16 of output), so that every access of a warp is contiguous (32768 x 7168: MX
// 88 us, 6.8 TB/s; NV 98).  Quantising is bound by integer and conversion
// instructions (8192 tokens to 4 experts each, K = 7168: MX 70 us, of which the
// bytes need 36, NV with a division per element 141; with the SwiGLU, 32768 x
// 2048, 79 and 103).  MX with 8 elements per thread took 100 us, so a thread
// takes 16, a whole NV block or half an MX one: what is done once per block is
// then done by one or two threads.  The rows are read with 32-byte loads where
// they are aligned to 32 bytes, else with two of 16; amax is taken on the 16-bit
// patterns, two at a time, where NaN and infinity order above every number (they
// mark the block's scale NaN); bf16 rows are scaled in pairs.  A team of threads
// takes a row, without divisions by the row length.
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
    int32_t team;        // threads per row
    const float* tensor_scale;
    uint8_t* codes;
    uint8_t* scales;
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void widen2(__nv_bfloat16, uint32_t u, float& lo, float& hi) {
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xFFFF0000u);
}
__device__ __forceinline__ void widen2(__half, uint32_t u, float& lo, float& hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    lo = f.x;
    hi = f.y;
}
template <typename T>
__device__ __forceinline__ void widen8(const uint4& u, float (&v)[8]) {
    widen2(T(), u.x, v[0], v[1]);
    widen2(T(), u.y, v[2], v[3]);
    widen2(T(), u.z, v[4], v[5]);
    widen2(T(), u.w, v[6], v[7]);
}
__device__ __forceinline__ float widen1(__nv_bfloat16, uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ float widen1(__half, uint32_t bits) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
// Bit pattern of infinity: magnitudes from here on are not numbers
template <typename T>
constexpr uint32_t kInf = 0x7F80u;
template <>
constexpr uint32_t kInf<__half> = 0x7C00u;

// Eight values times a power of two, as fp32.  bf16 pairs are multiplied as they
// are: the result is exact or too small to matter (below 2^-126, code 0).
__device__ __forceinline__ void scale8(__nv_bfloat16, const uint4& u, float inv, float (&v)[8]) {
    const __nv_bfloat162 f = __float2bfloat162_rn(inv);
    uint4 r;
    const uint32_t* a = &u.x;
    uint32_t* b = &r.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 m = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(a + j), f);
        b[j] = *reinterpret_cast<const uint32_t*>(&m);
    }
    widen8<__nv_bfloat16>(r, v);
}
__device__ __forceinline__ void scale8(__half, const uint4& u, float inv, float (&v)[8]) {
    widen8<__half>(u, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;
}

// Pieces of 16 elements that a thread has in flight (dequantising: 8 of 8)
constexpr int kPieces = 2;

// A team's row and the thread's place in it; false past the last row.
__device__ __forceinline__ bool team_row(int team, int64_t rows, int64_t& row, int& lane) {
    const int per = 256 / team;
    row = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / team;
    lane = threadIdx.x & (team - 1);
    return row < rows;
}

struct Piece {  // 16 elements
    uint4 a, b;
};
// WIDE: p is aligned to 32 bytes
template <bool WIDE>
__device__ __forceinline__ Piece load_piece(const void* p) {
    Piece r;
    if constexpr (WIDE) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w), "=r"(r.b.x), "=r"(r.b.y), "=r"(r.b.z),
                       "=r"(r.b.w)
                     : "l"(p)
                     : "memory");
    } else {
        r.a = __ldcg(static_cast<const uint4*>(p));
        r.b = __ldcg(static_cast<const uint4*>(p) + 1);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ uint4 swiglu8(const uint4& gate, const uint4& up) {
    float g[8], u[8];
    widen8<T>(gate, g);
    widen8<T>(up, u);
    uint4 r;
    uint32_t* h = &r.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = pack2(T(), silu(g[2 * j]) * u[2 * j], silu(g[2 * j + 1]) * u[2 * j + 1]);
    return r;
}

constexpr uint32_t kAbs = 0x7FFF7FFFu;
__device__ __forceinline__ uint32_t top_of(const uint4& u) {
    return max_u16x2(max_u16x2(u.x & kAbs, u.y & kAbs), max_u16x2(u.z & kAbs, u.w & kAbs));
}

template <typename T, bool NV, bool SWIGLU, bool WIDE>
__global__ void __launch_bounds__(256) k_quantize_fp4(const QuantArgs a) {
    pdl_trigger();
    pdl_wait();
    int64_t r;
    int me;
    const bool real = team_row(a.team, a.rows, r, me);  // all lanes stay for the shuffles
    const int pieces = a.K / 16, blocks = NV ? pieces : pieces / 2;
    const float g = NV && a.tensor_scale ? ld_dep(a.tensor_scale) : 1.0f;
    int64_t xr = r;
    bool have = real;
    if (real && a.src) {
        const int s = ld_dep(a.src + r);
        xr = s / a.src_div;
        have = s >= 0 && xr < a.x_rows;
    }
    const T* row = static_cast<const T*>(a.x) + (have ? xr * a.ldx : 0);
    uint8_t* scales = a.scales + (real ? r * a.stride : 0);
    uint2* codes = reinterpret_cast<uint2*>(a.codes + (real ? r * (a.K / 2) : 0));
    if (real)
        for (int i = blocks + me; i < a.stride; i += a.team) scales[i] = 0;  // the padding
    for (int p0 = 0; p0 < pieces; p0 += kPieces * a.team) {
        Piece in[kPieces], up[SWIGLU ? kPieces : 1];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = p0 + i * a.team + me;
            in[i].a = in[i].b = make_uint4(0, 0, 0, 0);
            if constexpr (SWIGLU) up[i] = in[i];
            if (have && p < pieces) {
                if constexpr (SWIGLU) {  // gate and up columns interleaved per 128
                    const T* q = row + (p >> 3) * 256 + (p & 7) * 16;
                    in[i] = load_piece<WIDE>(q);
                    up[i] = load_piece<WIDE>(q + 128);
                } else {
                    in[i] = load_piece<WIDE>(row + p * 16);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if (p0 + i * a.team >= pieces) break;  // the same for every team
            const int p = p0 + i * a.team + me;
            if constexpr (SWIGLU) {
                in[i].a = swiglu8<T>(in[i].a, up[i].a);
                in[i].b = swiglu8<T>(in[i].b, up[i].b);
            }
            uint32_t top2 = max_u16x2(top_of(in[i].a), top_of(in[i].b));
            if constexpr (!NV) top2 = max_u16x2(top2, __shfl_xor_sync(0xFFFFFFFFu, top2, 1));
            const uint32_t bits = max(top2 & 0xFFFFu, top2 >> 16);
            const bool bad = bits >= kInf<T>;  // a NaN or infinity: the whole block is NaN
            uint32_t code;
            float v[8];
            uint2 q = make_uint2(0, 0);
            if constexpr (NV) {
                code = f32_to_e4m3(fminf(widen1(T(), bits) / (g * 6.0f), 448.0f));
                const float s = e4m3_to_f32(code) * g;
                if (s > 0.0f && !bad) {
                    widen8<T>(in[i].a, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] /= s;
                    q.x = f32x8_to_e2m1(v);
                    widen8<T>(in[i].b, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] /= s;
                    q.y = f32x8_to_e2m1(v);
                }
                code = bad ? 0x7Fu : code;
            } else {
                // amax = 1.m * 2^(e - 127) <= 1.5 * 2^2 * 2^(code - 127)
                const uint32_t top = __float_as_uint(widen1(T(), bits));
                const int c = static_cast<int>(top >> 23) - ((top & 0x7FFFFFu) <= 0x400000u ? 2 : 1);
                code = top ? static_cast<uint32_t>(max(c, 0)) : 127u;
                const float inv = bad ? 0.0f : __uint_as_float((254u - code) << 23);  // 2^(127 - code)
                scale8(T(), in[i].a, inv, v);
                q.x = f32x8_to_e2m1(v);
                scale8(T(), in[i].b, inv, v);
                q.y = f32x8_to_e2m1(v);
                code = bad ? 0xFFu : code;
            }
            if (real && p < pieces) {
                if (NV || (me & 1) == 0) scales[NV ? p : p >> 1] = static_cast<uint8_t>(code);
                codes[p] = q;
            }
        }
    }
}

// value = e2m1 * scale (* g), one rounding each
template <typename T, bool NV>
__global__ void __launch_bounds__(256)
    k_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, int stride, int team,
                     const float* tensor_scale, T* out, int64_t ldo) {
    constexpr int kShare = NV ? 2 : 4;
    pdl_trigger();
    pdl_wait();
    int64_t r;
    int me;
    if (!team_row(team, rows, r, me)) return;
    const int pieces = K / 8;
    const float g = NV && tensor_scale ? ld_dep(tensor_scale) : 1.0f;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(codes + r * (K / 2));
    for (int p0 = 0; p0 < pieces; p0 += 8 * team) {
        uint32_t q[8], code[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = p0 + i * team + me;
            q[i] = p < pieces ? ld_dep(row + p) : 0u;
            code[i] = p < pieces ? ld_dep(scales + r * stride + p / kShare) : 0u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = p0 + i * team + me;
            if (p >= pieces) break;
            const float s = NV ? e4m3_to_f32(code[i]) : e8m0_to_f32(code[i]);
            uint32_t h[4], v[4];
            e2m1x8_to_f16x2(q[i], h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(h + j));
                v[j] = NV ? pack2(T(), f.x * s * g, f.y * s * g) : pack2(T(), f.x * s, f.y * s);
            }
            *reinterpret_cast<uint4*>(out + r * ldo + p * 8) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}

// Threads per row: an eighth of its pieces, rounded up to a power of two.
int team_of(int pieces) {
    int team = 8;
    while (team < 256 && team * 8 < pieces) team *= 2;
    return team;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status_t check_fp4(int32_t fmt, int64_t rows, int32_t K) {
    if (fmt != MOE_FP4_MX && fmt != MOE_FP4_NV)
        return set_last_error(MOE_ERR_INVALID_ARG, "format = %d is neither MX (0) nor NV (1)", fmt);
    if (rows < 0 || K <= 0) return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0 and K > 0");
    if (K % 32) return set_last_error(MOE_ERR_UNSUPPORTED, "K = %d is not a multiple of 32", K);
    if (K > kRaggedMaxDim) return set_last_error(MOE_ERR_UNSUPPORTED, "K = %d is more than 2^30", K);
    if (rows > (1ll << 30)) return set_last_error(MOE_ERR_UNSUPPORTED, "more than 2^30 rows");
    return MOE_OK;
}

int64_t blocks_for(int64_t rows, int team) { return (rows + 256 / team - 1) / (256 / team); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_fp4_scale_stride(int32_t fmt, int32_t K) {
    if ((fmt != MOE_FP4_MX && fmt != MOE_FP4_NV) || K <= 0 || K % 32 || K > kRaggedMaxDim) return 0;
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
    a.team = team_of(K / 16);
    const dim3 grid(static_cast<unsigned>(blocks_for(rows, a.team)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool nv = fmt == MOE_FP4_NV, wide = (reinterpret_cast<uintptr_t>(x) & 31) == 0 && ldx % 16 == 0;
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, st, a); };
    auto pick = [&](auto t) {
        using T = decltype(t);
        if (nv)
            return swiglu ? (wide ? go(k_quantize_fp4<T, true, true, true>) : go(k_quantize_fp4<T, true, true, false>))
                          : (wide ? go(k_quantize_fp4<T, true, false, true>) : go(k_quantize_fp4<T, true, false, false>));
        return swiglu ? (wide ? go(k_quantize_fp4<T, false, true, true>) : go(k_quantize_fp4<T, false, true, false>))
                      : (wide ? go(k_quantize_fp4<T, false, false, true>) : go(k_quantize_fp4<T, false, false, false>));
    };
    const cudaError_t e = dtype == MOE_DTYPE_BF16 ? pick(__nv_bfloat16()) : pick(__half());
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
    const int team = team_of(K / 8);
    const dim3 grid(static_cast<unsigned>(blocks_for(rows, team)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel, auto* o) {
        return launch_pdl(kernel, grid, dim3(256), 0, st, static_cast<const uint8_t*>(codes),
                          static_cast<const uint8_t*>(scales), rows, K, stride, team, tensor_scale, o, ldo);
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
