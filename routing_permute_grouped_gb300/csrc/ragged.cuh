// ragged.cuh -- what the grouped products on ragged row groups share: the
// launch description and the reading of the group offsets.
//
// Token rows are sorted by group (expert): group e owns rows
// [offsets[e], offsets[e + 1]) of the row-major operands, with any sizes,
// starts and gaps.  The offsets live on the device, so nothing of the launch
// depends on them.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace moe {

constexpr int kRaggedMaxGroups = 256;
constexpr uint32_t kRaggedBadGroup = 0x4u;  // MOE_DEVERR_SEGMENT

struct RaggedArgs {
    const int32_t* offsets;  // [E + 1]
    int32_t R, N, K, E;      // rows, output columns, sum length (wgrad: M is K here), groups
    const float* row_scale;  // [R] or null
    const float* x_scale;    // [1] or null: 4-bit rows' tensor scale
    const float* w_scale;    // [E] or null: 4-bit weights' tensor scales
    void* out;
    int64_t ldo;             // output row stride (elements)
    uint32_t* status;        // device error word, may be null
};

// Rows [x, y) of group e; empty and flagged when they do not lie in [0, R].
__device__ __forceinline__ int2 group_rows(const RaggedArgs& a, int e) {
    const int lo = ld_dep(a.offsets + e);
    const int hi = ld_dep(a.offsets + e + 1);
    if (lo < 0 || hi < lo || hi > a.R) {
        if (a.status) atomicOr(a.status, kRaggedBadGroup);
        return make_int2(0, 0);
    }
    return make_int2(lo, hi);
}

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }

// ---------------------------------------------------------- 4-bit values --
// Two e2m1 codes (low nibble first) -> two floats; every e2m1 value is an f16
// value.
__device__ __forceinline__ float2 e2m1x2_to_f32x2(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// The nearest e2m1 codes of two values (v0 in the low nibble), ties to even,
// saturating at +-6.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float v0, float v1) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(v1), "f"(v0));
    return r;
}
// Power-of-two block scale 2^(code - 127); code 255 is NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t code) {
    return __uint_as_float(code == 255u ? 0x7FC00000u : (code == 0u ? 0x00400000u : code << 23));
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
    const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(code));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

}  // namespace moe
