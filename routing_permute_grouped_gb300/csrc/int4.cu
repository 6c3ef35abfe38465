// int4.cu -- rows to and from unsigned 4-bit codes with group scales.
//
// A row's elements share, `group` (32, 64 or 128) at a time, one scale of the
// rows' 16-bit type and one zero point; the last group may be short:
//   value = (code - zero) * scale, code 0 .. 15
//   symmetric (no zero points): scale = amax / 7, zero = 8, codes 1 .. 15
//   with zero points: scale = (hi - lo) / 15 with lo = min(0, least) and hi =
//     max(0, largest), zero = -lo / scale rounded to 0 .. 15
// Quotients are rounded to integers, ties to even, the scale to its type first.
//
// Eight codes are a 32-bit word: element 2 i in bits 4 i, element 2 i + 1 in bits
// 16 + 4 i, so that one mask of a shifted word gives two neighbouring elements in
// the low bits of two 16-bit halves, which is how the product widens them.
//
// x / scale is t = x * r, r an approximate 1 / scale, with one Newton correction t +=
// (x - t scale) r.  A quotient of two 16-bit numbers is a half integer exactly, where
// the correction finds it exactly, or further from one than 2^-14 of its value, so
// the integer is that of the exact quotient.  (Scales of bf16 below 2^-120, whose
// reciprocal may overflow, and of f16 below its normal range, which may be off by more
// than a step in 2^10, go another way, with divisions.)
//
// A thread takes 32 elements, so that what is done once for a group of 128 (the
// exchange of its ends, the scale, the zero point) is done by four threads: with 8
// elements per thread that was most of the work (262144 x 1024, groups of 128 with zero
// points: 267 us quantising and 132 back where this takes 147 and 103, by events around
// single calls; the kernels by themselves 144 and 97).  64 bytes of a row
// go as two accesses of 32 where they are aligned to it, else as four of 16 (169 and 134,
// before the quantiser's registers were held to 48 for five blocks per SM, 160 to 148).
// Back is bound by HBM (6.6 TB/s); quantising, at 4.6 TB/s, by its instructions, 15 for an
// element of each lane, integer ones most.
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/moe.h"
#include "int4.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kPiece = 32;  // elements of a thread

struct Int4Args {
    const void* x;
    int64_t ldx;
    int64_t rows;
    int32_t pieces;  // of a row
    int32_t groups;
    int32_t shift;   // log2 of the pieces of a group
    int32_t team;    // threads per row
    uint4* codes;    // of a piece
    void* scales;
    uint8_t* zeros;  // or null
};

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static constexpr uint32_t kInf = 0x7F80u, kNan = 0x7FFFu;
    static constexpr float kLeast = 0x1p-120f;  // of a scale whose reciprocal is a number
};
template <>
struct Pair<__half> {
    using type = __half2;
    static constexpr uint32_t kInf = 0x7C00u, kNan = 0x7FFFu;
    static constexpr float kLeast = 0x1p-14f;  // of a scale with all its bits
};
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    using P = typename Pair<T>::type;
    const P m = __hmax2_nan(*reinterpret_cast<const P*>(&a), *reinterpret_cast<const P*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
template <typename T>
__device__ __forceinline__ float low_half(uint32_t u) {
    const unsigned short h = static_cast<unsigned short>(u);
    return to_float<T>(*reinterpret_cast<const T*>(&h));
}
template <typename T>
__device__ __forceinline__ uint32_t bits_of(float f) {
    const T t = from_float<T>(f);
    return *reinterpret_cast<const unsigned short*>(&t);
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// t rounded to an integer, ties to even, as the low bits of a float (|t| < 2^21)
constexpr uint32_t kIntBias = 0x4B400000u;  // 1.5 * 2^23
__device__ __forceinline__ uint32_t int_bits(float t) { return __float_as_uint(t + 12582912.0f); }

__device__ __forceinline__ float rcp_near(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 64 bytes; WIDE: aligned to 32
template <bool WIDE>
__device__ __forceinline__ void load64(const void* p, uint32_t (&r)[16]) {
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(r[8 * i]), "=r"(r[8 * i + 1]), "=r"(r[8 * i + 2]), "=r"(r[8 * i + 3]), "=r"(r[8 * i + 4]),
                           "=r"(r[8 * i + 5]), "=r"(r[8 * i + 6]), "=r"(r[8 * i + 7])
                         : "l"(static_cast<const char*>(p) + 32 * i)
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 v = ld_dep(static_cast<const uint4*>(p) + i);
            r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
        }
    }
}
template <bool WIDE>
__device__ __forceinline__ void store64(void* p, const uint32_t (&r)[16]) {
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(static_cast<char*>(p) + 32 * i), "r"(r[8 * i]),
                         "r"(r[8 * i + 1]), "r"(r[8 * i + 2]), "r"(r[8 * i + 3]), "r"(r[8 * i + 4]), "r"(r[8 * i + 5]),
                         "r"(r[8 * i + 6]), "r"(r[8 * i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            static_cast<uint4*>(p)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    }
}

template <typename T, bool ZEROS, bool WIDE>
__global__ void __launch_bounds__(256, 5) k_quantize_int4(const __grid_constant__ Int4Args a) {
    pdl_trigger();
    pdl_wait();
    const int me = threadIdx.x & (a.team - 1);
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / a.team) + threadIdx.x / a.team;
    const bool real = r < a.rows;  // all lanes stay for the shuffles
    const T* row = static_cast<const T*>(a.x) + (real ? r * a.ldx : 0);
    const int padded = a.groups << a.shift, per = 1 << a.shift;
    const int first = me & ~31;  // a team of more than a warp: its warps past the row's end have no turn
    for (int p0 = 0; p0 + first < padded; p0 += a.team) {
        const int p = p0 + me;
        const bool have = real && p < a.pieces;
        uint32_t v[16];
        if (have) {
            load64<WIDE>(row + p * kPiece, v);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0;
        }
        constexpr uint32_t kAbs = 0x7FFF7FFFu, kSigns = 0x80008000u;
        // symmetric: the largest magnitude's pattern, where infinity and NaN order above
        // numbers; else (largest, largest of the negated) as a pair, NaN if one is
        uint32_t ends = 0;
        if constexpr (ZEROS) {
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                hi = max2<T>(hi, v[i]);
                lo = max2<T>(lo, v[i] ^ kSigns);
            }
            ends = max2<T>(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) ends = max_u16x2(ends, v[i] & kAbs);
            ends = max(ends & 0xFFFFu, ends >> 16);
        }
        for (int o = 1; o < per; o <<= 1) {
            const uint32_t other = __shfl_xor_sync(kAll, ends, o);
            ends = ZEROS ? max2<T>(ends, other) : max(ends, other);
        }
        const bool bad = (ends & 0x7FFFu) >= Pair<T>::kInf || (ZEROS && (ends >> 16 & 0x7FFFu) >= Pair<T>::kInf);
        float lo = 0.0f;
        uint32_t scale;
        if constexpr (ZEROS) {
            const float hi = low_half<T>(ends);
            lo = -low_half<T>(ends >> 16);
            scale = bits_of<T>((0.5f * hi - 0.5f * lo) / 7.5f);  // halves: hi - lo may pass the range
        } else {
            scale = bits_of<T>(low_half<T>(ends) / 7.0f);
        }
        scale = bad ? Pair<T>::kNan : scale;
        const float s = low_half<T>(scale), inv = rcp_near(s);
        auto quotient = [&](float x) {
            const float t = x * inv;
            return fmaf(fmaf(-t, s, x), inv, t);
        };
        uint32_t zero = ZEROS ? 0u : 8u, word[4];
        if (s >= Pair<T>::kLeast) {
            // a scale within half a step of its quotient: |x| / scale is below 7.5, and
            // x / scale + zero is above -0.5 and below 16.5
            if constexpr (ZEROS) zero = min(int_bits(quotient(-lo)) - kIntBias, 15u);
            const float most = 15.0f - static_cast<float>(zero);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                word[w] = 0x11111111u * (zero - kIntBias);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t u = v[4 * w + (j >> 1)];
                    const float t = quotient(low_half<T>(j & 1 ? u >> 16 : u));
                    word[w] += int_bits(ZEROS ? fminf(t, most) : t) << (4 * (j >> 1) + 16 * (j & 1));
                }
            }
        } else {  // a scale of few bits, 0 or not a number
            const bool numbers = s > 0.0f;
            if (ZEROS && numbers) zero = min(int_bits(fminf(-lo / s, 15.0f)) - kIntBias, 15u);
            const float least = -static_cast<float>(zero), most = 15.0f + least;
#pragma unroll 1
            for (int w = 0; w < 4; ++w) {
                uint32_t sum = 0x11111111u * zero;
                if (numbers) {
                    sum -= 0x11111111u * kIntBias;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t u = w == 0 ? v[j >> 1] : w == 1 ? v[4 + (j >> 1)] : w == 2 ? v[8 + (j >> 1)] : v[12 + (j >> 1)];
                        const float t = low_half<T>(j & 1 ? u >> 16 : u) / s;
                        sum += int_bits(fminf(fmaxf(t, least), most)) << (4 * (j >> 1) + 16 * (j & 1));
                    }
                }
                if (w == 0) word[0] = sum;
                if (w == 1) word[1] = sum;
                if (w == 2) word[2] = sum;
                if (w == 3) word[3] = sum;
            }
        }
        if (have) a.codes[r * a.pieces + p] = make_uint4(word[0], word[1], word[2], word[3]);
        if (real && p < padded && (me & (per - 1)) == 0) {
            const int64_t at = r * a.groups + (p >> a.shift);
            static_cast<uint16_t*>(a.scales)[at] = static_cast<uint16_t>(scale);
            if constexpr (ZEROS) a.zeros[at] = static_cast<uint8_t>(zero);
        }
    }
}

// (code - zero) scale = ((128 + code) - (128 + zero)) scale: the difference is exact, and
// so is its product with a 16-bit scale in fp32.  (Two products and their difference, one
// operation less, pass fp32's range from bf16 scales of 2^121 on, which are a group's with
// elements from 1.7e37.)
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) k_dequantize_int4(const __grid_constant__ Int4Args a, T* out, int64_t ldo) {
    pdl_trigger();
    pdl_wait();
    const int me = threadIdx.x & (a.team - 1);
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / a.team) + threadIdx.x / a.team;
    if (r >= a.rows) return;
    for (int p = me; p < a.pieces; p += a.team) {
        const uint4 q = ld_dep(a.codes + r * a.pieces + p);
        const int64_t at = r * a.groups + (p >> a.shift);
        const float s = low_half<T>(ld_dep(static_cast<const uint16_t*>(a.scales) + at));
        const uint32_t z = a.zeros ? ld_dep(a.zeros + at) : 8u;
        const float back = -128.0f - static_cast<float>(z);
        const uint32_t word[4] = {q.x, q.y, q.z, q.w};
        uint32_t v[16];
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t u;  // 128 + code as the upper halves of two fp32 numbers
                asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(word[w] >> (4 * j)), "r"(0x000F000Fu), "r"(0x43004300u));
                v[4 * w + j] = pack2(T(), (__uint_as_float(u << 16) + back) * s, (__uint_as_float(u & 0xFFFF0000u) + back) * s);
            }
        store64<WIDE>(out + r * ldo + p * kPiece, v);
    }
}

// Threads per row: as many as its pieces, rounded up to a power of two, 4 to 256.
int team_of(int pieces) {
    int team = 4;
    while (team < 256 && team < pieces) team *= 2;
    return team;
}

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

moe_status_t check_int4(int32_t group, int32_t dtype, int64_t rows, int32_t K) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_last_error(MOE_ERR_INVALID_ARG, "dtype = %d is neither bf16 (0) nor f16 (1)", dtype);
    if (rows < 0) return set_last_error(MOE_ERR_INVALID_ARG, "rows must be >= 0");
    if (rows > (1ll << 30)) return set_last_error(MOE_ERR_UNSUPPORTED, "more than 2^30 rows");
    return static_cast<moe_status_t>(check_int4_row(group, K));
}

Int4Args args_of(int32_t group, int64_t rows, int32_t K, void* codes, void* scales, void* zeros) {
    Int4Args a{};
    a.rows = rows;
    a.pieces = K / kPiece;
    a.groups = (K + group - 1) / group;
    a.shift = group == 32 ? 0 : group == 64 ? 1 : 2;
    a.team = team_of(a.pieces);
    a.codes = static_cast<uint4*>(codes);
    a.scales = scales;
    a.zeros = static_cast<uint8_t*>(zeros);
    return a;
}

dim3 grid_of(const Int4Args& a) {
    const int per = 256 / a.team;
    return dim3(static_cast<unsigned>((a.rows + per - 1) / per));
}

}  // namespace

int check_int4_row(int32_t group, int32_t K) {
    if (group != 32 && group != 64 && group != 128)
        return set_last_error(MOE_ERR_UNSUPPORTED, "group = %d is none of 32, 64, 128", group);
    if (K <= 0) return set_last_error(MOE_ERR_INVALID_ARG, "K must be > 0");
    if (K % 32) return set_last_error(MOE_ERR_UNSUPPORTED, "K = %d is not a multiple of 32", K);
    if (K > kRaggedMaxDim) return set_last_error(MOE_ERR_UNSUPPORTED, "K = %d is more than 2^30", K);
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_quantize_int4(int32_t group, int32_t dtype, int64_t rows, int32_t K, const void* x,
                                          int64_t ldx, void* codes, void* scales, void* zeros, void* stream) {
    const moe_status_t s = check_int4(group, dtype, rows, K);
    if (s != MOE_OK) return s;
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 2))
        return set_last_error(MOE_ERR_INVALID_ARG, "x and codes must be 16-byte aligned, scales 2-byte");
    if (ldx < K || ldx % 8)
        return set_last_error(MOE_ERR_INVALID_ARG, "the row stride must cover the row and be a multiple of 8 elements");
    Int4Args a = args_of(group, rows, K, codes, scales, zeros);
    a.x = x;
    a.ldx = ldx;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = aligned(x, 32) && ldx % 16 == 0;
    auto go = [&](auto t, auto z) {
        using T = decltype(t);
        constexpr bool ZEROS = decltype(z)::value;
        return wide ? launch_pdl(k_quantize_int4<T, ZEROS, true>, grid_of(a), dim3(256), 0, st, a)
                    : launch_pdl(k_quantize_int4<T, ZEROS, false>, grid_of(a), dim3(256), 0, st, a);
    };
    auto by_type = [&](auto t) { return zeros ? go(t, std::true_type()) : go(t, std::false_type()); };
    const cudaError_t e = dtype == MOE_DTYPE_BF16 ? by_type(__nv_bfloat16()) : by_type(__half());
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit weights: %s", cudaGetErrorString(e));
}

extern "C" moe_status_t moe_dequantize_int4(int32_t group, int32_t dtype, int64_t rows, int32_t K, const void* codes,
                                            const void* scales, const void* zeros, void* out, int64_t ldo,
                                            void* stream) {
    const moe_status_t s = check_int4(group, dtype, rows, K);
    if (s != MOE_OK) return s;
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !out) return set_last_error(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned(codes, 16) || !aligned(scales, 2) || !aligned(out, 16))
        return set_last_error(MOE_ERR_INVALID_ARG, "codes and out must be 16-byte aligned, scales 2-byte");
    if (ldo < K || ldo % 8)
        return set_last_error(MOE_ERR_INVALID_ARG, "the row stride must cover the row and be a multiple of 8 elements");
    const Int4Args a = args_of(group, rows, K, const_cast<void*>(codes), const_cast<void*>(scales),
                               const_cast<void*>(zeros));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = aligned(out, 32) && ldo % 16 == 0;
    auto go = [&](auto* o) {
        using T = std::remove_pointer_t<decltype(o)>;
        return wide ? launch_pdl(k_dequantize_int4<T, true>, grid_of(a), dim3(256), 0, st, a, o, ldo)
                    : launch_pdl(k_dequantize_int4<T, false>, grid_of(a), dim3(256), 0, st, a, o, ldo);
    };
    const cudaError_t e = dtype == MOE_DTYPE_BF16 ? go(static_cast<__nv_bfloat16*>(out)) : go(static_cast<__half*>(out));
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit values: %s", cudaGetErrorString(e));
}
