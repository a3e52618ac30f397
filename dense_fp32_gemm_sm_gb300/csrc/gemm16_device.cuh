// gemm16_device.cuh -- activations of the 16-bit layers and their derivatives, in FP32, without
// branches and with two instructions of the special-function unit each.
//
// The factor that may be infinite is clamped where the other one is 0 (or the product below
// FP32's range), so that a pre-activation of -inf gives 0 and not 0 * inf.  A NaN stays one.
#pragma once

#include "mxfp4_device.cuh"

namespace fgemm {
namespace h16 {

using mx::after_previous_kernel;
using mx::from_float;
using mx::relu;
using mx::to_float;

// min and max that keep a NaN.
__device__ __forceinline__ float at_most(float x, float most)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(most));
    return r;
}

__device__ __forceinline__ float at_least(float x, float least)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(least));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float reciprocal_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// For a = |z|: e = exp(-a^2/2) and the normal tail q = Phi(-a) = e g(a).  g falls from 1/2 as 1/a: a
// polynomial in t = 1 / (1 + 0.31 a), the variable of Hastings' approximations (1955), its coefficients a
// minimax fit of the relative error for a up to 20 (1.7e-7; 5e-7 as evaluated in FP32).  Beyond 20 both
// are 0.  By normcdff the layer's epilogue took 1.3 times the whole product (8192 x 11008 x 4096, Z
// kept: 562 us against 431 without an activation).
__device__ __forceinline__ void normal_tail(float a, float &e, float &q)
{
    const float t = reciprocal_fast(fmaf(0.31f, a, 1.0f));
    e = exp2_fast(-0.721347520444482f * a * a);  // log2(e) / 2
    float g = fmaf(0.0359170846f, t, -0.141935625f);
    g = fmaf(g, t, 0.155671924f);
    g = fmaf(g, t, -0.0154948533f);
    g = fmaf(g, t, 0.110444422f);
    g = fmaf(g, t, 0.107662495f);
    g = fmaf(g, t, 0.124079033f);
    g = fmaf(g, t, 0.123655601f);
    q = e * (g * t);
}

// z Phi(z) = max(0, z) - |z| Phi(-|z|).
__device__ __forceinline__ float gelu(float z)
{
    const float a = at_most(fabsf(z), 20.0f);
    float e, q;
    normal_tail(a, e, q);
    return fmaf(-a, q, relu(z));
}

// Phi(z) + z phi(z): s for z < 0, 1 - s for z > 0, with s = Phi(-|z|) - |z| phi(z).
__device__ __forceinline__ float gelu_slope(float z)
{
    const float a = at_most(fabsf(z), 20.0f);
    float e, q;
    normal_tail(a, e, q);
    const float s = fmaf(a * -0.398942280401433f, e, q);
    return z > 0.0f ? 1.0f - s : s;
}

__device__ __forceinline__ float sigmoid(float z) { return reciprocal_fast(1.0f + exp2_fast(-1.44269504088896f * z)); }

__device__ __forceinline__ float silu(float z)
{
    z = at_least(z, -100.0f);
    return z * sigmoid(z);
}

__device__ __forceinline__ float silu_slope(float z)
{
    z = at_most(at_least(z, -100.0f), 100.0f);
    const float s = sigmoid(z);
    return s * fmaf(z, 1.0f - s, 1.0f);
}

// v act'(z).  ReLU's is a gate: what is behind a closed one, NaN included, does not matter.
__device__ __forceinline__ float through(float v, float z, int act)
{
    return act == FGEMM_ACT_RELU ? (z > 0.0f ? v : 0.0f)
           : act == FGEMM_ACT_GELU ? v * gelu_slope(z)
           : act == FGEMM_ACT_SILU ? v * silu_slope(z)
                                   : v;
}

// Two values to 16 bits, a in the low half.
template <class T> __device__ __forceinline__ uint32_t pack(float a, float b);
template <> __device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return reinterpret_cast<const uint32_t &>(v);
}
template <> __device__ __forceinline__ uint32_t pack<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return reinterpret_cast<const uint32_t &>(v);
}

}  // namespace h16
}  // namespace fgemm
