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
// x / scale is x * (1 / scale) with one Newton correction t += (x - t scale) /
// scale.  A quotient of two 16-bit numbers is a half integer exactly, where the
// correction finds it exactly, or further from one than 2^-14 of its value, so
// the integer is that of the exact quotient (scales below 2^-120, whose
// reciprocal may overflow, are divided by).
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "int4.h"
#include "internal.h"
#include "ragged.cuh"

namespace moe {

#define set_last_error(status, ...) static_cast<moe_status_t>(record_error(status, __VA_ARGS__))

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kFlight = 4;  // words that a thread has in flight

struct Int4Args {
    const void* x;
    int64_t ldx;
    int64_t rows;
    int32_t words;   // K / 8
    int32_t groups;  // per row
    int32_t shift;   // log2 of the words of a group
    int32_t team;    // threads per row
    uint32_t* codes;
    void* scales;
    uint8_t* zeros;  // or null
};

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static constexpr uint32_t kInf = 0x7F80u, kNan = 0x7FFFu;
};
template <>
struct Pair<__half> {
    using type = __half2;
    static constexpr uint32_t kInf = 0x7C00u, kNan = 0x7FFFu;
};
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    using P = typename Pair<T>::type;
    const P m = __hmax2(*reinterpret_cast<const P*>(&a), *reinterpret_cast<const P*>(&b));
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

template <typename T, bool ZEROS>
__global__ void __launch_bounds__(256) k_quantize_int4(const __grid_constant__ Int4Args a) {
    pdl_trigger();
    pdl_wait();
    const int me = threadIdx.x & (a.team - 1);
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / a.team) + threadIdx.x / a.team;
    const bool real = r < a.rows;  // all lanes stay for the shuffles
    const T* row = static_cast<const T*>(a.x) + (real ? r * a.ldx : 0);
    uint32_t* codes = a.codes + (real ? r * a.words : 0);
    const int64_t first = real ? r * a.groups : 0;
    const int padded = a.groups << a.shift, per = 1 << a.shift;
    for (int p0 = 0; p0 < padded; p0 += kFlight * a.team) {
        uint4 in[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int p = p0 + i * a.team + me;
            in[i] = real && p < a.words ? ld_dep(reinterpret_cast<const uint4*>(row) + p) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            if (p0 + i * a.team >= padded) break;  // the same for every team
            const int p = p0 + i * a.team + me;
            const uint32_t* v = &in[i].x;
            constexpr uint32_t kAbs = 0x7FFF7FFFu, kSigns = 0x80008000u;
            // the largest magnitude's pattern, where infinity and NaN order above
            // numbers, and (largest, largest of the negated) as a pair
            uint32_t top = max_u16x2(max_u16x2(v[0] & kAbs, v[1] & kAbs), max_u16x2(v[2] & kAbs, v[3] & kAbs));
            top = max(top & 0xFFFFu, top >> 16);
            uint32_t ends = 0;
            if constexpr (ZEROS) {
                uint32_t hi = max2<T>(max2<T>(v[0], v[1]), max2<T>(v[2], v[3]));
                uint32_t lo = max2<T>(max2<T>(v[0] ^ kSigns, v[1] ^ kSigns), max2<T>(v[2] ^ kSigns, v[3] ^ kSigns));
                ends = max2<T>(max2<T>(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632)), 0u);
            }
            for (int o = 1; o < per; o <<= 1) {
                top = max(top, __shfl_xor_sync(kAll, top, o));
                if constexpr (ZEROS) ends = max2<T>(ends, __shfl_xor_sync(kAll, ends, o));
            }
            const bool bad = top >= Pair<T>::kInf;
            float lo = 0.0f;
            uint32_t scale;
            if constexpr (ZEROS) {
                const float hi = low_half<T>(ends);
                lo = -low_half<T>(ends >> 16);
                scale = bits_of<T>((0.5f * hi - 0.5f * lo) / 7.5f);  // halves: hi - lo may pass the range
            } else {
                scale = bits_of<T>(low_half<T>(top) / 7.0f);
            }
            scale = bad ? Pair<T>::kNan : scale;
            const float s = low_half<T>(scale);
            uint32_t zero = ZEROS ? 0u : 8u, word = 0;
            const bool numbers = s > 0.0f;
            if constexpr (ZEROS)
                if (numbers) zero = min(int_bits(-lo / s) - kIntBias, 15u);
            const float least = -static_cast<float>(zero), most = 15.0f + least, inv = 1.0f / s;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x0 = low_half<T>(v[j]), x1 = low_half<T>(v[j] >> 16);
                float t0 = x0 * inv, t1 = x1 * inv;
                t0 = fmaf(fmaf(-t0, s, x0), inv, t0);
                t1 = fmaf(fmaf(-t1, s, x1), inv, t1);
                if (s < 0x1p-120f) {
                    t0 = x0 / s;
                    t1 = x1 / s;
                }
                word += int_bits(fminf(fmaxf(t0, least), most)) << (4 * j);
                word += int_bits(fminf(fmaxf(t1, least), most)) << (16 + 4 * j);
            }
            word += 0x11111111u * (zero - kIntBias);
            if (!numbers) word = 0x11111111u * zero;
            if (real && p < a.words) codes[p] = word;
            if (real && p < padded && (me & (per - 1)) == 0) {
                static_cast<uint16_t*>(a.scales)[first + (p >> a.shift)] = static_cast<uint16_t>(scale);
                if constexpr (ZEROS) a.zeros[first + (p >> a.shift)] = static_cast<uint8_t>(zero);
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_dequantize_int4(const __grid_constant__ Int4Args a, T* out, int64_t ldo) {
    pdl_trigger();
    pdl_wait();
    const int me = threadIdx.x & (a.team - 1);
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / a.team) + threadIdx.x / a.team;
    if (r >= a.rows) return;
    const uint32_t* codes = a.codes + r * a.words;
    const int64_t first = r * a.groups;
    for (int p0 = 0; p0 < a.words; p0 += kFlight * a.team) {
        uint32_t q[kFlight], s[kFlight], z[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int p = p0 + i * a.team + me;
            const bool in = p < a.words;
            q[i] = in ? ld_dep(codes + p) : 0u;
            s[i] = in ? ld_dep(static_cast<const uint16_t*>(a.scales) + first + (p >> a.shift)) : 0u;
            z[i] = a.zeros && in ? ld_dep(a.zeros + first + (p >> a.shift)) : 8u;
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int p = p0 + i * a.team + me;
            if (p >= a.words) break;
            const float f = low_half<T>(s[i]), zero = static_cast<float>(z[i]);
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = pack2(T(), (static_cast<float>(q[i] >> (4 * j) & 15u) - zero) * f,
                             (static_cast<float>(q[i] >> (16 + 4 * j) & 15u) - zero) * f);
            *reinterpret_cast<uint4*>(out + r * ldo + p * 8) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}

// Threads per row: a kFlight-th of its words, at least a group of 128.
int team_of(int words) {
    int team = 16;
    while (team < 256 && team * kFlight < words) team *= 2;
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
    a.words = K / 8;
    a.groups = (K + group - 1) / group;
    a.shift = group == 32 ? 2 : group == 64 ? 3 : 4;
    a.team = team_of(a.words);
    a.codes = static_cast<uint32_t*>(codes);
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
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid_of(a), dim3(256), 0, st, a); };
    const cudaError_t e = dtype == MOE_DTYPE_BF16
                              ? (zeros ? go(k_quantize_int4<__nv_bfloat16, true>) : go(k_quantize_int4<__nv_bfloat16, false>))
                              : (zeros ? go(k_quantize_int4<__half, true>) : go(k_quantize_int4<__half, false>));
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
    const cudaError_t e =
        dtype == MOE_DTYPE_BF16
            ? launch_pdl(k_dequantize_int4<__nv_bfloat16>, grid_of(a), dim3(256), 0, st, a,
                         static_cast<__nv_bfloat16*>(out), ldo)
            : launch_pdl(k_dequantize_int4<__half>, grid_of(a), dim3(256), 0, st, a, static_cast<__half*>(out), ldo);
    return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "4-bit values: %s", cudaGetErrorString(e));
}
