// The e4m3 block format of the 8-bit floating point path, and its device helpers.
//
// Values are held as e4m3 codes (sign, 4 exponent bits, 3 mantissa bits, largest
// 448, no infinity) with one f32 scale per block of 128 along the reduction (the
// last block of a row may be shorter): activations one scale per row and block,
// weights one per 128 rows and block.  Quantizing a block:
//   a = max(max|v|, 2^-100)      (a NaN is passed over by the maximum)
//   code = e4m3(v * fl(448 / a)) (nearest even; |v| <= a, so nothing saturates
//                                 but by the rounding of the factor; NaN stays NaN)
//   scale = fl(a / 448)
// The floor keeps 448 / a finite and makes a block of zeros an ordinary one.  One
// reciprocal factor per block instead of a division per value: the f32 rounding
// of the factor and of the product move a value by 2^-23 of itself against a
// code's own half step of 2^-4, so a code differs from that of the real quotient
// only where the quotient lies that close to the middle of two codes.  A block
// with an infinity has scale infinity and NaN for every value it stands for.
#pragma once

#include <cuda_fp8.h>

#include "qg_common.cuh"

namespace qg {

constexpr int EB = 128;  // values per scale

__host__ __device__ constexpr int64_t e4m3_blocks(int64_t k) { return (k + EB - 1) / EB; }

// A block's largest magnitude, not below the floor.
__device__ __forceinline__ float e4m3_floor(float a) { return fmaxf(a, 0x1p-100f); }

// max over the warp of non-negative floats, none of them NaN: their bit patterns
// order as unsigned integers.
__device__ __forceinline__ float warp_max_nonneg(float a)
{
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
}

// Two codes, lo in bits 0-7.
__device__ __forceinline__ uint32_t e4m3_pack2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d)
{
    return e4m3_pack2(a, b) | (e4m3_pack2(c, d) << 16);
}

__device__ __forceinline__ float max_abs4(float4 v)
{
    // fmaxf passes over NaN; four NaN leave 0
    return fmaxf(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))), 0.0f);
}

// Four stream values (f32, or bf16 widened exactly).
template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
    using raw = float4;
    static __device__ __forceinline__ float4 widen(raw v) { return v; }
    static __device__ __forceinline__ raw narrow(float4 v) { return v; }
    static __device__ __forceinline__ float max_abs(raw v) { return max_abs4(v); }
};
template <>
struct Vec4<__nv_bfloat16> {
    using raw = uint2;
    static __device__ __forceinline__ float4 widen(raw v)
    {
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xffff0000u));
    }
    static __device__ __forceinline__ raw narrow(float4 v)
    {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    // two at a time; like fmaxf the packed maximum passes over NaN
    static __device__ __forceinline__ float max_abs(raw v)
    {
        const __nv_bfloat162 m = __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162 *>(&v.x)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&v.y)));
        return fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.0f);
    }
};

// SiLU(g) * u = g u / (1 + e^-g), zero where e^-g is beyond f32 (g <= -88.722).  The
// exponent is carried as a rounded product -x log2(e) and its remainder (an FMA, and the
// constant's own second part), so that the error of e^-x does not grow with |x|: the
// approximations of 2^y and 1/y are what is left of it.  They are a choice: at most 2^-21.5
// of the value over g in [-87, 100] (2^-23.7 in the mean square), and with expf and an IEEE
// division 2^-22.1 (2^-24.3), far below a code's half step of 2^-4 either way, but those
// take 17 % longer (15 us at 2048x9216x2560's 84, 1.3 at 512x3584x1024's 8.8).
// Both sides of the quotient carry the factor c, a little over a quarter: 1/y of a y
// beyond 2^126 is flushed to zero, and c (1 + e^-g) gets there only where e^-g is within
// 2^-10 of f32's end, 2^128.  x is g held at -88.7224, inside that last bit: whatever g's
// size below, e^-x is finite and the quotient a zero.
constexpr float kLog2e = 1.4426950216293335f;       // log2(e) rounded to f32
constexpr float kLog2eRest = 1.925963033500011e-08f;  // and what that leaves
constexpr float kLn2 = 0.693147181f;
constexpr float kSiluRange = 88.7224f;  // e^88.7224 = 2^128 (1 - 0.00044)
constexpr float kSiluC = 0.25f * (1.0f + 0x1p-10f);

__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float silu_mul_e(float g, float u)
{
    const float x = fminf(fmaxf(g, -kSiluRange), kSiluRange);
    const float hi = x * -kLog2e;
    const float rest = fmaf(x, kLog2eRest, fmaf(x, kLog2e, hi));  // x log2(e) + hi
    float e = ex2_approx(hi);
    e = fmaf(e, rest * -kLn2, e);
    return g * kSiluC * rcp_approx(fmaf(e, kSiluC, kSiluC)) * u;
}

}  // namespace qg
