// gemm16_device.cuh -- activations of the 16-bit layers and their derivatives, in FP32, two values at a time
// where the arithmetic counts: sm_103a has FP32 instructions of two lanes, and a chunk of 16 rows
// through GELU's slope was bound by its 40 instructions an element.
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

// ---- 16-bit values -------------------------------------------------------------------------

// The value of 16 bits (the low half of a word).
template <class T> __device__ __forceinline__ float from_bits(uint32_t bits);
template <> __device__ __forceinline__ float from_bits<__nv_bfloat16>(uint32_t bits) { return __uint_as_float(bits << 16); }
template <> __device__ __forceinline__ float from_bits<__half>(uint32_t bits)
{
    const uint16_t low = (uint16_t)bits;
    return __half2float(reinterpret_cast<const __half &>(low));
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

// ---- FP32, one and two at a time ------------------------------------------------------------

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

// 1/2 + a b, held in 0 .. 1.
__device__ __forceinline__ float half_and(float a, float b)
{
    float r;
    asm("fma.rn.sat.f32 %0, %1, %2, 0f3F000000;" : "=f"(r) : "f"(a), "f"(b));
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

struct Two {
    uint64_t bits;
};

__device__ __forceinline__ Two two(float a, float b)
{
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.bits) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ Two both(float x) { return two(x, x); }

__device__ __forceinline__ void split(Two x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.bits));
}

__device__ __forceinline__ Two fma(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits), "l"(c.bits));
    return r;
}

__device__ __forceinline__ Two mul(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.bits) : "l"(a.bits), "l"(b.bits));
    return r;
}

template <int N>
__device__ __forceinline__ Two polynomial(const float (&c)[N], Two x)
{
    Two h = both(c[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) h = fma(h, x, both(c[i]));
    return h;
}

__device__ __forceinline__ Two exp2_fast(Two x)
{
    float a, b;
    split(x, a, b);
    return two(exp2_fast(a), exp2_fast(b));
}

__device__ __forceinline__ Two reciprocal_fast(Two x)
{
    float a, b;
    split(x, a, b);
    return two(reciprocal_fast(a), reciprocal_fast(b));
}

// exp(-x^2 / 2).
__device__ __forceinline__ Two bell(Two x) { return exp2_fast(mul(mul(both(-0.721347520444482f), x), x)); }

// ---- GELU -----------------------------------------------------------------------------------

// z Phi(z) = max(0, z) - a q for a = |z| and the normal tail q = Phi(-a) = exp(-a^2/2) g(a).  g falls from 1/2
// as 1/a: a polynomial (TAIL times t) in t = 1 / (1 + 0.31 a), the variable of Hastings' approximations
// (1955), its coefficients a minimax fit of the relative error for a up to 20 (1.9e-7; 5e-7 as evaluated in
// FP32, 6.5e-7 where the reciprocal is a unit off).  From 20 on q is 0.  (By normcdff the layer's epilogue took
// 1.3 times the whole product: 8192 x 11008 x 4096, Z kept, 562 us against 431 without an activation.)
__device__ constexpr float TAIL[] = {0.0359170846f, -0.141935625f, 0.155671924f, -0.0154948533f,
                                     0.110444422f,  0.107662495f,  0.124079033f, 0.123655601f};

__device__ __forceinline__ void gelu(float &z0, float &z1)
{
    const Two a = two(at_most(fabsf(z0), 20.0f), at_most(fabsf(z1), 20.0f));
    const Two t = reciprocal_fast(fma(a, both(0.31f), both(1.0f))), q = mul(bell(a), mul(polynomial(TAIL, t), t));
    split(fma(mul(a, both(-1.0f)), q, two(relu(z0), relu(z1))), z0, z1);
}

// The slope Phi(z) + z phi(z), with Phi(z) = 1/2 + z P(2 z^2 / 5.5^2 - 1) for |z| up to 5.5, beyond which Phi is 0 or
// 1 to within FP32's rounding: P (CDF) is a Chebyshev fit of this even function, off by less than 1e-8, its
// coefficients add up to 0.4, and Phi as evaluated is 1.6e-8 off on average, 9e-8 at most.  (A gradient is
// rounded to 16 bits, to the other side the more often the less exact it is.  By the tail above it is up to 3.3e-7 off,
// and the weights' gradient of 2048 rows was twice as far off.)
__device__ constexpr float CDF[] = {0.000118079995f, -0.000285676331f, 0.000183916665f, -0.000356754608f, 0.00140742643f, -0.00265870243f,
                                    0.00407412974f,  -0.00665067835f,  0.0104686385f,   -0.015062524f,    0.0203073174f,  -0.0260361508f,
                                    0.0320769101f,   -0.0387937948f,   0.0477373339f,   -0.0641723126f,   0.12855193f};

__device__ __forceinline__ Two gelu_slope(float z0, float z1)
{
    const float c0 = at_least(at_most(z0, 5.5f), -5.5f), c1 = at_least(at_most(z1, 5.5f), -5.5f);
    const Two c = two(c0, c1);
    float p0, p1;
    split(polynomial(CDF, fma(mul(c, c), both(2.0f / (5.5f * 5.5f)), both(-1.0f))), p0, p1);
    // At -5.5 the halves' sum is -1.5e-8 (at 5.5 it rounds to 1): held in 0 .. 1, it is 0 from there on, and the slope ends with the
    // bell.  (A NaN becomes 0 here, and is back by c.)
    return fma(c, mul(both(0.398942280401433f), bell(two(z0, z1))), two(half_and(c0, p0), half_and(c1, p1)));
}

// The same by the tail: 1/2 - (1/2 - s) for z < 0, 1/2 + (1/2 - s) for z > 0, with s = Phi(-|z|) - |z| phi(z),
// off by 3.3e-7 at most; fewer operations.
__device__ __forceinline__ float gelu_slope_near(float z)
{
    const float a = at_most(fabsf(z), 20.0f), t = reciprocal_fast(fmaf(0.31f, a, 1.0f));
    float g = TAIL[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) g = fmaf(g, t, TAIL[i]);
    // exp(-a^2/2) (g t - a / sqrt(2 pi))
    const float s = exp2_fast(-0.721347520444482f * a * a) * fmaf(g, t, -0.398942280401433f * a);
    return 0.5f + copysignf(0.5f - s, z);
}

// ---- SiLU -----------------------------------------------------------------------------------

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

// ---- gradients ------------------------------------------------------------------------------

// ReLU's gradient is a gate: what is behind a closed one, NaN included, does not matter.
__device__ __forceinline__ float gate(float v, float z) { return z > 0.0f ? v : 0.0f; }

// act'(z) (GELU, SiLU) as its definition reads, each step rounded to nearest; a few units in the last place off.
static __device__ __noinline__ float slope_by_definition(float z, int act)
{
    if (act == FGEMM_ACT_GELU) {
        const float cdf = __fmul_rn(0.5f, erfcf(__fmul_rn(-z, 0.707106781186548f)));
        const float w = at_least(at_most(z, 20.0f), -20.0f);  // (0 * inf)
        return __fadd_rn(cdf, __fmul_rn(__fmul_rn(w, expf(__fmul_rn(__fmul_rn(-0.5f, z), z))), 0.398942280401433f));
    }
    const float c = at_least(at_most(z, 80.0f), -80.0f), s = __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-c)));
    return __fmul_rn(s, __fadd_rn(1.0f, __fmul_rn(c, __fadd_rn(1.0f, -s))));
}

// v act'(z) of two values, and the pair rounded to T as when act' is evaluated by its definition in FP32: by the fast
// evaluation where all values within both evaluations' errors round alike, else by the definition (one
// BF16 element in 1500).  GELU's slope is off by 3.3e-7 and 1.3e-7 at most, SiLU's by (1 + |z|) times 1.1e-7 in
// both; the bracket is about twice their sum.  (By gelu_slope, as the products do, the error is the definition's, 2.8e-8 and
// 2.5e-8 in the 2-norm over normal arguments; the tail's is 5.6e-8.  This is agreement with that order of operations.)
template <class T, int ACT>
__device__ __forceinline__ uint32_t through_exactly(float &v0, float &v1, float z0, float z1)
{
    if (ACT == FGEMM_ACT_NONE) return pack<T>(v0, v1);
    if (ACT == FGEMM_ACT_RELU) {
        v0 = gate(v0, z0);
        v1 = gate(v1, z1);
        return pack<T>(v0, v1);
    }
    const bool gelu = ACT == FGEMM_ACT_GELU;
    const float w0 = gelu ? 8.5e-7f : fmaf(at_most(fabsf(z0), 80.0f), 5e-7f, 5e-7f), g0 = fabsf(v0);
    const float w1 = gelu ? 8.5e-7f : fmaf(at_most(fabsf(z1), 80.0f), 5e-7f, 5e-7f), g1 = fabsf(v1);
    // (Not to be contracted with a sum that they go into: column sums are the same with D and without.)
    const float f0 = __fmul_rn(v0, gelu ? gelu_slope_near(z0) : silu_slope(z0));
    const float f1 = __fmul_rn(v1, gelu ? gelu_slope_near(z1) : silu_slope(z1));
    const uint32_t d = pack<T>(fmaf(-w0, g0, f0), fmaf(-w1, g1, f1)), differ = d ^ pack<T>(fmaf(w0, g0, f0), fmaf(w1, g1, f1));
    if (differ != 0) {
        v0 = differ & 0xFFFFu ? __fmul_rn(v0, slope_by_definition(z0, ACT)) : f0;
        v1 = differ >> 16 ? __fmul_rn(v1, slope_by_definition(z1, ACT)) : f1;
        return pack<T>(v0, v1);
    }
    v0 = f0;
    v1 = f1;
    return d;
}

}  // namespace h16
}  // namespace fgemm
