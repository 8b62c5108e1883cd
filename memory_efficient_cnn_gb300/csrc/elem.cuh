// Element types of the row operators (feed-forward, norms, gradient clipping):
// conversion to and from fp32, 16-byte vectors, and the activations.
#pragma once

#include <atomic>
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

// Lets a kernel have up to `bytes` (always the same for it) of dynamic shared memory. Once for each
// device: asking takes longer than a launch.
template <auto Kernel>
inline cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---- activations of the gated feed-forward, and their derivatives at g

// The standard normal distribution at g.
__device__ __forceinline__ float normal_cdf(float g) { return 0.5f * erfcf(-0.70710678118654752f * g); }
__device__ __forceinline__ float sigmoid_f32(float g) { return 1.0f / (1.0f + expf(-g)); }
// (1 + tanh z) / 2 is the sigmoid of 2 z; this is 2 z for gelu_tanh's z.
__device__ __forceinline__ float gelu_tanh_arg(float g) { return 1.5957691216057307f * (g + 0.044715f * g * g * g); }

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    if (ACT == IM2WIN_ACT_SILU) return g * sigmoid_f32(g);
    if (ACT == IM2WIN_ACT_GELU) return g * normal_cdf(g);
    if (ACT == IM2WIN_ACT_GELU_TANH) return g * sigmoid_f32(gelu_tanh_arg(g));
    if (ACT == IM2WIN_ACT_RELU) return g < 0.0f ? 0.0f : g;
    return sigmoid_f32(g);
}

// a = act(g), d = act'(g)
template <int ACT>
__device__ __forceinline__ void act_both(float g, float &a, float &d) {
    if (ACT == IM2WIN_ACT_GELU) {
        const float p = normal_cdf(g);
        a = g * p;
        d = fmaf(g, expf(-0.5f * g * g) * 0.39894228040143268f, p);
    } else if (ACT == IM2WIN_ACT_RELU) {
        a = act_value<IM2WIN_ACT_RELU>(g);
        d = g > 0.0f ? 1.0f : 0.0f;
    } else {
        const float p = sigmoid_f32(ACT == IM2WIN_ACT_GELU_TANH ? gelu_tanh_arg(g) : g);
        a = ACT == IM2WIN_ACT_SIGMOID ? p : g * p;
        const float s = a * (1.0f - p);
        // (g^2 is bounded, so that 0 times it stays 0)
        d = ACT == IM2WIN_ACT_SIGMOID ? s
            : ACT == IM2WIN_ACT_SILU  ? p + s
                                      : fmaf(s, 1.5957691216057307f * fmaf(0.134145f, fminf(g * g, 1e38f), 1.0f), p);
    }
}

// The same for results that are rounded to 16 bits, two values at a time: sums
// and products by the paired fp32 instructions, exponentials and reciprocals by
// the hardware's approximations (about 1e-6 off in all, a five-hundredth of
// fp16's rounding). The epilogues of short products are bound by these
// instructions: gelu over 200704 x 512 hidden values took 215 us at 32
// instructions a value.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float both) { return f2(both, both); }
__device__ __forceinline__ void split(F2 a, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
template <typename Fn>
__device__ __forceinline__ F2 each2(F2 a, Fn f) {
    float lo, hi;
    split(a, lo, hi);
    return f2(f(lo), f(hi));
}
__device__ __forceinline__ F2 exp2_2(F2 a) {
    return each2(a, [](float v) {
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v));
        return v;
    });
}
__device__ __forceinline__ F2 recip2(F2 a) {
    return each2(a, [](float v) {
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(v));
        return v;
    });
}

// gelu's normal distribution: erfc(z) = t P(t) exp(-z^2), t = 1 / (1 + 0.38 z), the
// form of Hastings' rational approximations (Abramowitz and Stegun, 7.1.23 to
// 7.1.28), with a P of degree 6 fitted here by minimax least squares over
// 0 <= z <= 12: relative error at most 1.04e-6, also in the tail. The
// coefficients below are halved and negative. This is minus its part beyond size =
// |g| standard deviations; e is exp(-g^2 / 2).
__device__ __forceinline__ F2 minus_normal_tail2(F2 g, F2 size, F2 &e) {
    e = exp2_2(mul2(mul2(g, f2(-0.72134752044448170f)), g));  // -log2(e) / 2
    const F2 t = recip2(fma2(size, f2(0.38f * 0.70710678118654752f), f2(1.0f)));
    F2 q = f2(0.062708848354241800f);
    q = fma2(q, t, f2(-0.16801843157332533f));
    q = fma2(q, t, f2(0.034957064694897890f));
    q = fma2(q, t, f2(-0.12391755923373703f));
    q = fma2(q, t, f2(-0.09029702208545247f));
    q = fma2(q, t, f2(-0.10828872910161622f));
    q = fma2(q, t, f2(-0.10714365505117787f));
    return mul2(mul2(q, t), e);
}

// The factor of g in act(g) (act(g) itself for sigmoid, the step for relu); e is
// exp(-g^2 / 2) for gelu.
template <int ACT>
__device__ __forceinline__ F2 act_factor2(F2 g, F2 &e) {
    if (ACT == IM2WIN_ACT_GELU) {
        const F2 tail = minus_normal_tail2(g, each2(g, [](float v) { return fabsf(v); }), e);
        float g0, g1, t0, t1, c0, c1;
        split(g, g0, g1);
        split(tail, t0, t1);
        split(add2(tail, f2(1.0f)), c0, c1);
        return f2(g0 < 0.0f ? -t0 : c0, g1 < 0.0f ? -t1 : c1);
    }
    if (ACT == IM2WIN_ACT_RELU) return each2(g, [](float v) { return v > 0.0f ? 1.0f : 0.0f; });
    F2 arg;
    if (ACT == IM2WIN_ACT_GELU_TANH)  // -log2(e) 2 sqrt(2 / pi) (g + 0.044715 g^3)
        arg = mul2(g, fma2(mul2(g, g), f2(-0.10294324f), f2(-2.3022082f)));
    else
        arg = mul2(g, f2(-1.4426950408889634f));
    return recip2(add2(exp2_2(arg), f2(1.0f)));
}

template <int ACT>
__device__ __forceinline__ F2 act_value2(F2 g) {
    if (ACT == IM2WIN_ACT_RELU) return each2(g, [](float v) { return v < 0.0f ? 0.0f : v; });
    F2 e;
    if (ACT == IM2WIN_ACT_GELU) {  // max(g, 0) - |g| tail, which needs no selection (bounded: 0 times it stays 0)
        const F2 size = each2(g, [](float v) { return fminf(fabsf(v), 1e30f); });
        const F2 tail = minus_normal_tail2(g, size, e);
        return fma2(size, tail, each2(g, [](float v) { return fmaxf(v, 0.0f); }));
    }
    const F2 p = act_factor2<ACT>(g, e);
    return ACT == IM2WIN_ACT_SIGMOID ? p : mul2(g, p);
}

// a = act(g), d = act'(g)
template <int ACT>
__device__ __forceinline__ void act_both2(F2 g, F2 &a, F2 &d) {
    F2 e;
    const F2 p = act_factor2<ACT>(g, e);
    if (ACT == IM2WIN_ACT_RELU) {
        a = act_value2<ACT>(g);
        d = p;
        return;
    }
    a = ACT == IM2WIN_ACT_SIGMOID ? p : mul2(g, p);
    if (ACT == IM2WIN_ACT_GELU) {
        d = fma2(g, mul2(e, f2(0.39894228040143268f)), p);
        return;
    }
    const F2 s = mul2(a, fma2(p, f2(-1.0f), f2(1.0f)));
    if (ACT == IM2WIN_ACT_SIGMOID) d = s;
    if (ACT == IM2WIN_ACT_SILU) d = add2(p, s);
    if (ACT == IM2WIN_ACT_GELU_TANH) {
        const F2 sq = each2(mul2(g, g), [](float v) { return fminf(v, 1e38f); });  // (0 times it stays 0)
        d = fma2(s, fma2(sq, f2(0.21406859f), f2(1.5957691f)), p);
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
