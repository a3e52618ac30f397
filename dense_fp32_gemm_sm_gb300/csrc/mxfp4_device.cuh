// mxfp4_device.cuh -- device helpers of the MXFP4 kernels: element types, scales, codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mxfp4.h"

namespace fgemm {
namespace mx {

// See mxfp4_launch.h: wait for the kernel before this one, then let the next one come.
__device__ __forceinline__ void after_previous_kernel()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

template <class T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// max(0, x); a NaN stays, as what a spoiled block reaches is not a number.
__device__ __forceinline__ float relu(float x)
{
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
    return r;
}

// A block's scale byte from the bits of its largest magnitude (the exponent field, less
// the 2 of the largest code's exponent); 255 when the block holds a NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t largest_bits)
{
    const uint32_t e = largest_bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^(127 - s), the factor that brings a block into the codes' range (s <= 252, so the
// factor and, but for results far below half the smallest code, the products are exact).
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - min(s, 252u)) << 23); }

// 2^(s - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t s)
{
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7FFFFFFFu : s << 23);
}

// Eight values to eight codes, x[0] in the low nibble; nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8])
{
    uint32_t r;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n"
        "}\n"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// Eight codes to their values (before the scale).
__device__ __forceinline__ void decode8(uint32_t codes, float (&x)[8])
{
    uint32_t h[4];
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n"
        "}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The two codes of a byte to their values.
__device__ __forceinline__ float2 decode2(uint32_t byte)
{
    uint32_t h;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %1;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "}\n"
        : "=r"(h)
        : "r"(byte));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace mx
}  // namespace fgemm
