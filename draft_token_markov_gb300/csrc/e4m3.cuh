// e4m3.cuh -- conversions between e4m3 and the 16-bit types, four elements at a
// time, and what a cache's scales are taken from.
#pragma once
#include <cstdint>

#include <cuda_fp16.h>

namespace dtm {

constexpr float kE4m3Max = 448.0f;
constexpr float kLeastScale = 9.094947017729282e-13f;   // 2^-40: of a block of zeros

// Two e4m3 values in the low half of x, as fp16: exact.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t x) {
    uint32_t r;
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(x));
    return r;
}
// Four of them.
__device__ __forceinline__ void f16x4_of_e4m3(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
__device__ __forceinline__ float2 f32x2_of_e4m3(uint32_t x) {
    const uint32_t h = f16x2_of_e4m3(x);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Four values rounded to nearest, ties to even; beyond +-448 they become +-448,
// NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_of_f32(float a, float b, float c, float d) {
    uint32_t r;
    asm("{ .reg .b16 l, h; cvt.rn.satfinite.e4m3x2.f32 l, %2, %1; cvt.rn.satfinite.e4m3x2.f32 h, %4, %3; mov.b32 %0, {l, "
        "h}; }"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The least power of two that max / 448 is not above, 2^-40 at least: 448 is 1.75
// * 2^8.
__device__ __forceinline__ float scale_of(float max) {
    const uint32_t b = __float_as_uint(max);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);
    return fmaxf(__uint_as_float((uint32_t)::max(e, 1) << 23), kLeastScale);
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

// ------------------------------------------------- of the attention kernels

// A weight is 2^(y - m + kShiftE4), m lagging behind the maximum by kLazyE4 at most:
// up to 2^15 in fp16, so that small ones stay normal.
constexpr float kLazyE4 = 8.0f, kShiftE4 = 7.0f;

// log2 of a value's scale, which enters the exponent of its weight.
__device__ __forceinline__ float scale_log2(float s) { return __log2f(fmaxf(s, 8.673617379884035e-19f /* 2^-60 */)); }

// The exponent of the power of two that brings a row's largest element just below
// 2^14: BF16 queries times that become fp16 ones without a loss.
__device__ __forceinline__ int row_exponent(float max) {
    const int e = max > 0.0f ? min((int)(__float_as_uint(max) >> 23), 254) : 127;
    return min(127 + 13 - e, 100);
}
__device__ __forceinline__ float power_of_two(int k) { return __uint_as_float((uint32_t)(127 + k) << 23); }

__device__ __forceinline__ bool usable_scale(float s) { return s > 0.0f && s < INFINITY; }

}  // namespace dtm
