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

__device__ __forceinline__ float sigmoid_f32(float g) { return 1.0f / (1.0f + expf(-g)); }

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    if (ACT == IM2WIN_ACT_SILU) return g * sigmoid_f32(g);
    if (ACT == IM2WIN_ACT_GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));
    if (ACT == IM2WIN_ACT_GELU_TANH)
        return 0.5f * g * (1.0f + tanhf(0.79788456080286536f * (g + 0.044715f * g * g * g)));
    if (ACT == IM2WIN_ACT_RELU) return g > 0.0f ? g : (g != g ? g : 0.0f);
    return sigmoid_f32(g);
}

// a = act(g), d = act'(g)
template <int ACT>
__device__ __forceinline__ void act_both(float g, float &a, float &d) {
    if (ACT == IM2WIN_ACT_SILU) {
        const float p = sigmoid_f32(g);
        a = g * p;
        d = p + a * (1.0f - p);
    } else if (ACT == IM2WIN_ACT_GELU) {
        const float cdf = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
        a = g * cdf;
        d = cdf + g * expf(-0.5f * g * g) * 0.39894228040143268f;
    } else if (ACT == IM2WIN_ACT_GELU_TANH) {
        const float t = tanhf(0.79788456080286536f * (g + 0.044715f * g * g * g));
        a = 0.5f * g * (1.0f + t);
        d = 0.5f * (1.0f + t) + 0.5f * g * (1.0f - t * t) * 0.79788456080286536f *
                                      (1.0f + 0.134145f * fminf(g * g, 1e38f));  // (bounded: 0 times it stays 0)
    } else if (ACT == IM2WIN_ACT_RELU) {
        a = act_value<IM2WIN_ACT_RELU>(g);
        d = g > 0.0f ? 1.0f : 0.0f;
    } else {
        a = sigmoid_f32(g);
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
