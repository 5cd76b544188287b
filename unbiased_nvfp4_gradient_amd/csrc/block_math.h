// block_math.h -- the activations of a feed-forward block and their derivatives, in FP32.
#pragma once
#include "train_device.h"

namespace nvfp4t {

enum { NONE = 0, RELU = 1, GELU = 2, GELU_TANH = 3, SILU = 4 };   // NVFP4_ACT_*

// 1 / (1 + e^-x), from 2^(-x log2 e): the exponential takes |x| 2^-24 relative from its argument's
// rounding; below -88 it is 0.
__device__ __forceinline__ float sigmoid(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * x));
}

// tanh's argument in gelu_tanh, doubled: z (1 + tanh(u)) / 2 = z sigmoid(2 u).
__device__ __forceinline__ float tanh_argument(float z)
{
    return 1.59576912160573071176f * __builtin_fmaf(0.044715f * z * z, z, z);
}

// e^(-z^2 / 2) and the normal distribution's lower part: the upper part of a = |z| is
// e^(-a^2 / 2) times a polynomial in 1 / (1 + 0.304 a), fitted to erfcx(a / sqrt 2) / 2 over [0, 14]
// with the least largest relative error (10^-7; 3.5 10^-7 with the roundings of its evaluation).
__device__ __forceinline__ void normal(float z, float &density, float &lower)
{
    const float a = fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.304f, a, 1.0f));
    float s = 0.036624159663915634f;
    s = __builtin_fmaf(s, t, -0.1543489545583725f);
    s = __builtin_fmaf(s, t, 0.19059546291828156f);
    s = __builtin_fmaf(s, t, -0.041701145470142365f);
    s = __builtin_fmaf(s, t, 0.12281636148691177f);
    s = __builtin_fmaf(s, t, 0.10264070332050323f);
    s = __builtin_fmaf(s, t, 0.12213654816150665f);
    s = __builtin_fmaf(s, t, 0.12123686075210571f);
    density = __builtin_amdgcn_exp2f(-0.72134752044448170368f * z * z);
    const float upper = s * t * density;
    lower = z < 0.0f ? upper : 1.0f - upper;
}

template <int ACT> __device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == RELU) return z < 0.0f ? 0.0f : z;             // NaN stays
    else if constexpr (ACT == SILU) return z * sigmoid(z);
    else if constexpr (ACT == GELU_TANH) return z * sigmoid(tanh_argument(z));
    else if constexpr (ACT == GELU) {
        float density, lower;
        normal(z, density, lower);
        return z * lower;
    } else return z;
}

// The activation and its derivative.  Beyond +-100 every derivative is 0 or 1 in FP32: its terms take
// z from inside, so that none is 0 times infinity.
template <int ACT> __device__ __forceinline__ void activate2(float z, float &value, float &slope)
{
    const float c = fminf(fmaxf(z, -100.0f), 100.0f);
    if constexpr (ACT == RELU) {
        value = z < 0.0f ? 0.0f : z;
        slope = z <= 0.0f ? 0.0f : 1.0f;
    } else if constexpr (ACT == SILU) {
        const float s = sigmoid(z);
        value = z * s;
        slope = s * __builtin_fmaf(c, 1.0f - s, 1.0f);
    } else if constexpr (ACT == GELU_TANH) {
        const float s = sigmoid(tanh_argument(z));
        value = z * s;
        const float du = __builtin_fmaf(0.21406444881780076f * c, c, 1.59576912160573071176f);
        slope = s * __builtin_fmaf(c * (1.0f - s), du, 1.0f);
    } else if constexpr (ACT == GELU) {
        float density, lower;
        normal(z, density, lower);
        value = z * lower;
        slope = __builtin_fmaf(c * 0.39894228040143267794f, density, lower);
    } else {
        value = z;
        slope = 1.0f;
    }
}

}  // namespace nvfp4t
