// gemm16_device.cuh -- activations of the 16-bit layers and their derivatives, in FP32.
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

// Phi(z) by normcdff: 1 + erff(z / sqrt 2) would cancel below z = -3, where Phi is what 16 bits
// still resolve.
__device__ __forceinline__ float gelu(float z) { return fmaxf(z, -20.0f) * normcdff(z); }

__device__ __forceinline__ float gelu_slope(float z)
{
    const float density = 0.398942280401432678f * __expf(-0.5f * z * z);
    return fmaf(fminf(fmaxf(z, -20.0f), 20.0f), density, normcdff(z));
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

__device__ __forceinline__ float silu(float z) { return fmaxf(z, -100.0f) * sigmoid(z); }

__device__ __forceinline__ float silu_slope(float z)
{
    const float s = sigmoid(z);
    return s * fmaf(fminf(fmaxf(z, -100.0f), 100.0f), 1.0f - s, 1.0f);
}

__device__ __forceinline__ float activate(float z, int act)
{
    return act == FGEMM_ACT_RELU ? relu(z) : act == FGEMM_ACT_GELU ? gelu(z) : act == FGEMM_ACT_SILU ? silu(z) : z;
}

// v act'(z).  ReLU's is a gate: what is behind a closed one, NaN included, does not matter.
__device__ __forceinline__ float through(float v, float z, int act)
{
    return act == FGEMM_ACT_RELU ? (z > 0.0f ? v : 0.0f)
           : act == FGEMM_ACT_GELU ? v * gelu_slope(z)
           : act == FGEMM_ACT_SILU ? v * silu_slope(z)
                                   : v;
}

}  // namespace h16
}  // namespace fgemm
