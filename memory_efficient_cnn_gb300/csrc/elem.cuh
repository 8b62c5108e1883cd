// Element types of the row operators (feed-forward, norms, gradient clipping):
// conversion to and from fp32, 16-byte vectors, and the activations.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "im2win_internal.cuh"

namespace im2win {

using bf16_t = __nv_bfloat16;
using f16_t = __half;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(f16_t v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(bf16_t v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ f16_t from_f32<f16_t>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
    return __float2bfloat16_rn(v);
}

// V elements moved as one aligned word.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    static constexpr int N = V;
    T v[V];
};
template <typename T>
using Vec16 = Vec<T, 16 / (int)sizeof(T)>;

// Calls f with a null pointer of the C++ type of dtype code `dtype`; false for
// an unknown code.
template <typename Fn>
inline bool with_dtype(int dtype, Fn f) {
    switch (dtype) {
        case IM2WIN_F32: f((float *)nullptr); return true;
        case IM2WIN_F16: f((f16_t *)nullptr); return true;
        case IM2WIN_BF16: f((bf16_t *)nullptr); return true;
        default: return false;
    }
}

inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---- activations of the gated feed-forward, and their derivatives at g
//
// FAST is for results that are rounded to 16 bits: exponentials and quotients by
// the hardware's approximations (about 1e-6 off, a five-hundredth of fp16's
// rounding), and the normal distribution's tail by the polynomial below. With
// them the epilogues of the products no longer cost more than the products:
// gelu over 200704 x 512 hidden values took 221 us with erff and expf.

template <bool FAST>
__device__ __forceinline__ float exp_f32(float v) {
    return FAST ? __expf(v) : expf(v);
}
template <bool FAST>
__device__ __forceinline__ float recip_f32(float v) {
    return FAST ? __fdividef(1.0f, v) : 1.0f / v;
}
template <bool FAST>
__device__ __forceinline__ float sigmoid_f32(float g) {
    return recip_f32<FAST>(1.0f + exp_f32<FAST>(-g));
}

// The standard normal distribution at g, and its density.
// FAST: erfc(z) = t P(t) exp(-z^2), t = 1 / (1 + 0.38 z), the form of Hastings'
// rational approximations (Abramowitz and Stegun, 7.1.23 to 7.1.28), with a P of
// degree 6 fitted here by minimax least squares over 0 <= z <= 12: relative error
// at most 1.04e-6, also in the tail.
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float g, float &density) {
    const float e = exp_f32<FAST>(-0.5f * g * g);
    density = e * 0.39894228040143268f;
    if (!FAST) return 0.5f * erfcf(-0.70710678118654752f * g);
    const float t = recip_f32<FAST>(fmaf(0.38f * 0.70710678118654752f, fabsf(g), 1.0f));
    float q = -0.12541769670848360f;
    q = fmaf(q, t, 0.33603686314665066f);
    q = fmaf(q, t, -0.06991412938979578f);
    q = fmaf(q, t, 0.24783511846747405f);
    q = fmaf(q, t, 0.18059404117089478f);
    q = fmaf(q, t, 0.21657745820323432f);
    q = fmaf(q, t, 0.21428731011020574f);
    const float tail = 0.5f * q * t * e;
    return g < 0.0f ? tail : 1.0f - tail;
}

// Twice the argument of gelu_tanh's tanh: (1 + tanh z) / 2 is the sigmoid of 2 z.
__device__ __forceinline__ float gelu_tanh_arg(float g) { return 1.5957691216057307f * (g + 0.044715f * g * g * g); }

template <int ACT, bool FAST>
__device__ __forceinline__ float act_value(float g) {
    if (ACT == IM2WIN_ACT_SILU) return g * sigmoid_f32<FAST>(g);
    if (ACT == IM2WIN_ACT_GELU) {
        float density;
        return g * normal_cdf<FAST>(g, density);
    }
    if (ACT == IM2WIN_ACT_GELU_TANH) return g * sigmoid_f32<FAST>(gelu_tanh_arg(g));
    if (ACT == IM2WIN_ACT_RELU) return g > 0.0f ? g : (g != g ? g : 0.0f);
    return sigmoid_f32<FAST>(g);
}

// a = act(g), d = act'(g)
template <int ACT, bool FAST>
__device__ __forceinline__ void act_both(float g, float &a, float &d) {
    if (ACT == IM2WIN_ACT_SILU) {
        const float p = sigmoid_f32<FAST>(g);
        a = g * p;
        d = fmaf(a, 1.0f - p, p);
    } else if (ACT == IM2WIN_ACT_GELU) {
        float density;
        const float p = normal_cdf<FAST>(g, density);
        a = g * p;
        d = fmaf(g, density, p);
    } else if (ACT == IM2WIN_ACT_GELU_TANH) {
        const float p = sigmoid_f32<FAST>(gelu_tanh_arg(g));
        a = g * p;
        // (g^2 is bounded, so that 0 times it stays 0)
        d = fmaf(a * (1.0f - p), 1.5957691216057307f * fmaf(0.134145f, fminf(g * g, 1e38f), 1.0f), p);
    } else if (ACT == IM2WIN_ACT_RELU) {
        a = act_value<IM2WIN_ACT_RELU, FAST>(g);
        d = g > 0.0f ? 1.0f : 0.0f;
    } else {
        a = sigmoid_f32<FAST>(g);
        d = a * (1.0f - a);
    }
}

// Calls f with an integral constant of a run-time activation code; false for an
// unknown one.
template <int V>
struct IntC {
    static constexpr int value = V;
};
template <typename Fn>
inline bool with_act(int act, Fn f) {
    switch (act) {
        case IM2WIN_ACT_SILU: f(IntC<IM2WIN_ACT_SILU>()); return true;
        case IM2WIN_ACT_GELU: f(IntC<IM2WIN_ACT_GELU>()); return true;
        case IM2WIN_ACT_GELU_TANH: f(IntC<IM2WIN_ACT_GELU_TANH>()); return true;
        case IM2WIN_ACT_RELU: f(IntC<IM2WIN_ACT_RELU>()); return true;
        case IM2WIN_ACT_SIGMOID: f(IntC<IM2WIN_ACT_SIGMOID>()); return true;
        default: return false;
    }
}

// The same on the device.
template <typename Fn>
__device__ __forceinline__ void with_act_device(int act, Fn f) {
    switch (act) {
        case IM2WIN_ACT_SILU: f(IntC<IM2WIN_ACT_SILU>()); break;
        case IM2WIN_ACT_GELU: f(IntC<IM2WIN_ACT_GELU>()); break;
        case IM2WIN_ACT_GELU_TANH: f(IntC<IM2WIN_ACT_GELU_TANH>()); break;
        case IM2WIN_ACT_RELU: f(IntC<IM2WIN_ACT_RELU>()); break;
        default: f(IntC<IM2WIN_ACT_SIGMOID>()); break;
    }
}

}  // namespace im2win
