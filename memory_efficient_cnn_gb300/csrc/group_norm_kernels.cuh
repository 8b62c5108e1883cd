// Group norm with its activation, channels last:
//   xh = (x - mean) i,  z = xh w + b,  y = act(z)
// with the mean and inverse deviation i of the P D elements of an image's group, and
//   dz = dy act'(z),  db = sum dz,  dw = sum dz xh  (over images and positions),
//   dx = i (w dz - m1 - xh m2),  m1, m2: the group's means of w dz and w dz xh.
//
// The pass over positions works by channel: a thread keeps to one vector of channels, so
// that neither the alignment of groups to vectors nor their size matters, and leaves a
// mean and a sum of squared deviations for each channel and chunk of positions. These
// join by n1 n2 / (n1 + n2) (m1 - m2)^2 (Chan, Golub, LeVeque), without the cancellation
// of a sum of squares.
#pragma once

#include "group_norm.cuh"
#include "tc_ptx.cuh"

namespace im2win {
namespace gnorm {
namespace {

template <int BYTES>
struct WordOf;
template <>
struct WordOf<16> { using type = uint4; };
template <>
struct WordOf<8> { using type = uint2; };
template <>
struct WordOf<4> { using type = uint32_t; };
template <>
struct WordOf<2> { using type = uint16_t; };

// V elements as they lie in memory, and as pairs of fp32 (V = 1: the upper one is zero).
template <typename T, int V>
struct Group {
    static constexpr int PAIRS = (V + 1) / 2;
    using Word = typename WordOf<V * (int)sizeof(T)>::type;
};
template <typename T, int V>
__device__ __forceinline__ void to_pairs(const typename Group<T, V>::Word &word, F2 (&v)[Group<T, V>::PAIRS]) {
    if constexpr (sizeof(T) == 4) {
        const float *f = reinterpret_cast<const float *>(&word);
        if constexpr (V == 1) {
            v[0] = f2(f[0], 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
        }
    } else if constexpr (V == 1) {
        v[0] = f2(to_f32(*reinterpret_cast<const T *>(&word)), 0.0f);
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&word);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (std::is_same_v<T, bf16_t>) {
                v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[i] = f2(f.x, f.y);
            }
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ typename Group<T, V>::Word from_pairs(const F2 (&v)[Group<T, V>::PAIRS]) {
    typename Group<T, V>::Word word;
    if constexpr (sizeof(T) == 4) {
        float *f = reinterpret_cast<float *>(&word);
#pragma unroll
        for (int i = 0; i < (V + 1) / 2; ++i) {
            float lo, hi;
            split(v[i], lo, hi);
            f[2 * i] = lo;
            if (V > 1) f[2 * i + 1] = hi;
        }
    } else if constexpr (V == 1) {
        float lo, hi;
        split(v[0], lo, hi);
        *reinterpret_cast<T *>(&word) = from_f32<T>(lo);
    } else {
        uint32_t *w = reinterpret_cast<uint32_t *>(&word);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float lo, hi;
            split(v[i], lo, hi);
            w[i] = tc::pack2(lo, hi, std::is_same_v<T, bf16_t>);
        }
    }
    return word;
}

template <typename Fn>
__device__ __forceinline__ void with_norm_act(int act, Fn f) {
    if (act == IM2WIN_ACT_NONE) f(IntC<IM2WIN_ACT_NONE>());
    else with_act_device(act, f);
}
// act(z); fp32 by the functions themselves, 16-bit types by the approximations made for them.
template <typename T, int ACT>
__device__ __forceinline__ F2 act_of(F2 z) {
    if constexpr (ACT == IM2WIN_ACT_NONE) return z;
    else if constexpr (sizeof(T) == 4) return each2(z, [](float v) { return act_value<ACT>(v); });
    else return act_value2<ACT>(z);
}
// act'(z)
template <typename T, int ACT>
__device__ __forceinline__ F2 slope_of(F2 z) {
    if constexpr (ACT == IM2WIN_ACT_NONE) {
        return f2(1.0f);
    } else if constexpr (sizeof(T) == 4) {
        return each2(z, [](float v) {
            float a, d;
            act_both<ACT>(v, a, d);
            return d;
        });
    } else {
        F2 a, d;
        act_both2<ACT>(z, a, d);
        return d;
    }
}
__device__ __forceinline__ F2 neg2(F2 a) { return mul2(a, f2(-1.0f)); }

// What a thread of the position passes works on.
template <typename T, int V>
struct Place {
    using Word = typename Group<T, V>::Word;
    int64_t n, p0, p1, base;  // image, positions of the block, element (n, 0, channel)
    int chunk, slab, row, col, c;  // c: first channel of the thread's vector
    bool in;
    __device__ explicit Place(const GroupArgs &a) {
        int64_t id = blockIdx.x;
        chunk = (int)(id % a.chunks);
        id /= a.chunks;
        slab = (int)(id % a.slabs);
        n = id / a.slabs;
        row = threadIdx.x / a.cols, col = threadIdx.x % a.cols;
        c = (slab * a.cols + col) * V;
        in = row < a.rows && c < a.C;
        p0 = chunk * a.len, p1 = min(a.P, p0 + a.len);
        base = n * a.P * a.C + c;
    }
    __device__ const Word *at(const void *x, const GroupArgs &a, int64_t p) const {
        return reinterpret_cast<const Word *>(static_cast<const T *>(x) + base + p * a.C);
    }
    __device__ Word *at(void *x, const GroupArgs &a, int64_t p) const {
        return reinterpret_cast<Word *>(static_cast<T *>(x) + base + p * a.C);
    }
};

// The thread's channels' parameters and statistics.
template <typename T, int V>
struct Channels {
    static constexpr int PAIRS = Group<T, V>::PAIRS;
    F2 mean[PAIRS], inv[PAIRS], w[PAIRS], b[PAIRS];
    __device__ Channels(const GroupArgs &a, int64_t n, int c) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float v[4][2] = {};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (2 * i + j >= V) continue;
                const int ch = c + 2 * i + j;
                const float2 s = reinterpret_cast<const float2 *>(a.stats)[n * a.G + ch / a.D];
                v[0][j] = s.x, v[1][j] = s.y;
                v[2][j] = a.w ? to_f32(static_cast<const T *>(a.w)[ch]) : 1.0f;
                v[3][j] = a.b ? to_f32(static_cast<const T *>(a.b)[ch]) : 0.0f;
            }
            mean[i] = f2(v[0][0], v[0][1]), inv[i] = f2(v[1][0], v[1][1]);
            w[i] = f2(v[2][0], v[2][1]), b[i] = f2(v[3][0], v[3][1]);
        }
    }
    __device__ F2 hat(int i, F2 x) const { return mul2(add2(x, neg2(mean[i])), inv[i]); }
};

// Means and sums of squared deviations of a chunk's positions, for each channel.
template <typename T, int V>
__global__ void __launch_bounds__(THREADS) gn_moments(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    __shared__ F2 red[2 * PAIRS][THREADS];
    const Place<T, V> at(a);
    tc::allow_dependents();
    tc::grid_dependency_wait();
    F2 mean[PAIRS], m2[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) mean[i] = m2[i] = f2(0.0f);
    float count = 0.0f;
    // joins another set of values' moments to the thread's
    auto join = [&](float n, auto other) {
        const float total = count + n, share = n / total, scale = count * share;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            F2 om, o2;
            other(i, om, o2);
            const F2 d = add2(om, neg2(mean[i]));
            mean[i] = fma2(d, f2(share), mean[i]);
            m2[i] = fma2(mul2(d, d), f2(scale), add2(m2[i], o2));
        }
        count = total;
    };
    if (at.in) {
        for (int64_t p = at.p0 + at.row; p < at.p1; p += (int64_t)a.rows * BATCH) {
            Word word[BATCH];
            int n = 0;
#pragma unroll
            for (int j = 0; j < BATCH; ++j)
                if (p + (int64_t)j * a.rows < at.p1) word[j] = *at.at(a.x, a, p + (int64_t)j * a.rows), n = j + 1;
            F2 sum[PAIRS], sq[PAIRS];
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) sum[i] = sq[i] = f2(0.0f);
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                if (j >= n) continue;
                F2 v[PAIRS];
                to_pairs<T, V>(word[j], v);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) sum[i] = add2(sum[i], v[i]);
            }
            const float inv = 1.0f / n;
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) sum[i] = mul2(sum[i], f2(inv));
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                if (j >= n) continue;
                F2 v[PAIRS];
                to_pairs<T, V>(word[j], v);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    const F2 d = add2(v[i], neg2(sum[i]));
                    sq[i] = fma2(d, d, sq[i]);
                }
            }
            join((float)n, [&](int i, F2 &om, F2 &o2) { om = sum[i], o2 = sq[i]; });
        }
    }
    // over the block's rows, in halves
    auto count_of = [&](int row) { return row >= at.p1 - at.p0 ? 0.0f : (float)((at.p1 - at.p0 - row + a.rows - 1) / a.rows); };
    __shared__ float counts[THREADS];
    if (at.col == 0 && at.row < a.rows) counts[at.row] = count_of(at.row);
    for (int n = a.rows; n > 1;) {
        const int h = (n + 1) / 2;
        if (at.in && at.row >= h && at.row < n) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) red[2 * i][threadIdx.x] = mean[i], red[2 * i + 1][threadIdx.x] = m2[i];
        }
        __syncthreads();
        const float other = at.row < n - h ? counts[at.row + h] : 0.0f;
        if (at.in && other > 0.0f) {
            const int t = threadIdx.x + h * a.cols;
            join(other, [&](int i, F2 &om, F2 &o2) { om = red[2 * i][t], o2 = red[2 * i + 1][t]; });
        }
        __syncthreads();
        if (at.col == 0 && at.row < n - h) counts[at.row] += other;
        n = h;
        __syncthreads();
    }
    if (at.in && at.row == 0) {
        float *m = a.part + (at.n * a.chunks + at.chunk) * a.C + at.c, *q = m + a.N * a.chunks * a.C;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float lo, hi, lo2, hi2;
            split(mean[i], lo, hi);
            split(m2[i], lo2, hi2);
            m[2 * i] = lo, q[2 * i] = lo2;
            if (V > 1) m[2 * i + 1] = hi, q[2 * i + 1] = hi2;
        }
    }
}

// Sum over SPAN threads (a warp, or the block), the same for each and in a fixed order.
template <int SPAN>
__device__ __forceinline__ float span_sum(float v, float *s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (SPAN == 32) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < SPAN / 32; ++i) t += s[i];
    __syncthreads();
    return t;
}

// A group's chunks and channels become its mean and inverse deviation; SPAN threads a group.
template <int SPAN>
__global__ void __launch_bounds__(THREADS) gn_stats(const __grid_constant__ GroupArgs a) {
    __shared__ float s[THREADS / 32];
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t id = (int64_t)blockIdx.x * (THREADS / SPAN) + threadIdx.x / SPAN;
    if (id >= a.N * a.G) return;
    const int64_t n = id / a.G, half = a.N * a.chunks * a.C;
    const int c0 = (int)(id % a.G) * a.D, items = a.D * a.chunks;
    const float *m = a.part + n * a.chunks * a.C + c0;
    // chunk k holds count(k) positions
    auto count = [&](int k) { return (float)(min(a.P, (k + 1) * a.len) - k * a.len); };
    float sum = 0.0f;
    for (int i = threadIdx.x % SPAN; i < items; i += SPAN) {
        const int k = i / a.D;
        sum = fmaf(m[(int64_t)k * a.C + i - k * a.D], count(k), sum);
    }
    const float total = (float)a.P * a.D, mean = span_sum<SPAN>(sum, s) / total;
    float sq = 0.0f;
    for (int i = threadIdx.x % SPAN; i < items; i += SPAN) {
        const int k = i / a.D;
        const int64_t at = (int64_t)k * a.C + i - k * a.D;
        const float d = m[at] - mean;
        sq += fmaf(d * d, count(k), m[half + at]);
    }
    sq = span_sum<SPAN>(sq, s);
    if (threadIdx.x % SPAN == 0) reinterpret_cast<float2 *>(a.stats)[id] = make_float2(mean, 1.0f / sqrtf(sq / total + a.eps));
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS) gn_apply(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    const Place<T, V> at(a);
    tc::allow_dependents();
    tc::grid_dependency_wait();
    if (!at.in) return;
    const Channels<T, V> ch(a, at.n, at.c);
    with_norm_act(a.act, [&](auto kind) {
        for (int64_t p = at.p0 + at.row; p < at.p1; p += a.rows * 4) {
            Word word[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (p + j * a.rows < at.p1) word[j] = *at.at(a.x, a, p + j * a.rows);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (p + j * a.rows >= at.p1) continue;
                F2 v[PAIRS];
                to_pairs<T, V>(word[j], v);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) v[i] = act_of<T, decltype(kind)::value>(fma2(ch.hat(i, v[i]), ch.w[i], ch.b[i]));
                *at.at(a.y, a, p + j * a.rows) = from_pairs<T, V>(v);
            }
        }
    });
}

// Sums of dz and dz xh over a chunk's positions, for each channel.
template <typename T, int V>
__global__ void __launch_bounds__(THREADS) gn_back_sums(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS, FEW = BATCH / 2;
    using Word = typename Group<T, V>::Word;
    __shared__ F2 red[2 * PAIRS][THREADS];
    const Place<T, V> at(a);
    tc::allow_dependents();
    tc::grid_dependency_wait();
    F2 s0[PAIRS], s1[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) s0[i] = s1[i] = f2(0.0f);
    if (at.in) {
        const Channels<T, V> ch(a, at.n, at.c);
        with_norm_act(a.act, [&](auto kind) {
            for (int64_t p = at.p0 + at.row; p < at.p1; p += a.rows * FEW) {
                Word wx[FEW], wd[FEW];
#pragma unroll
                for (int j = 0; j < FEW; ++j)
                    if (p + j * a.rows < at.p1) wx[j] = *at.at(a.x, a, p + j * a.rows), wd[j] = *at.at(a.dy, a, p + j * a.rows);
#pragma unroll
                for (int j = 0; j < FEW; ++j) {
                    if (p + j * a.rows >= at.p1) continue;
                    F2 x[PAIRS], d[PAIRS];
                    to_pairs<T, V>(wx[j], x);
                    to_pairs<T, V>(wd[j], d);
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        const F2 hat = ch.hat(i, x[i]);
                        const F2 dz = mul2(d[i], slope_of<T, decltype(kind)::value>(fma2(hat, ch.w[i], ch.b[i])));
                        s0[i] = add2(s0[i], dz);
                        s1[i] = fma2(dz, hat, s1[i]);
                    }
                }
            }
        });
    }
    for (int n = a.rows; n > 1;) {
        const int h = (n + 1) / 2;
        if (at.in && at.row >= h && at.row < n) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) red[2 * i][threadIdx.x] = s0[i], red[2 * i + 1][threadIdx.x] = s1[i];
        }
        __syncthreads();
        if (at.in && at.row < n - h) {
            const int t = threadIdx.x + h * a.cols;
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) s0[i] = add2(s0[i], red[2 * i][t]), s1[i] = add2(s1[i], red[2 * i + 1][t]);
        }
        __syncthreads();
        n = h;
    }
    if (at.in && at.row == 0) {
        float *m = a.part + (at.n * a.chunks + at.chunk) * a.C + at.c, *q = m + a.N * a.chunks * a.C;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float lo, hi, lo2, hi2;
            split(s0[i], lo, hi);
            split(s1[i], lo2, hi2);
            m[2 * i] = lo, q[2 * i] = lo2;
            if (V > 1) m[2 * i + 1] = hi, q[2 * i + 1] = hi2;
        }
    }
}

// A group's means of w dz and w dz xh; SPAN threads a group.
template <typename T, int SPAN>
__global__ void __launch_bounds__(THREADS) gn_back_means(const __grid_constant__ GroupArgs a) {
    __shared__ float s[THREADS / 32];
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t id = (int64_t)blockIdx.x * (THREADS / SPAN) + threadIdx.x / SPAN;
    if (id >= a.N * a.G) return;
    const int64_t n = id / a.G, half = a.N * a.chunks * a.C;
    const int c0 = (int)(id % a.G) * a.D, items = a.D * a.chunks;
    const float *m = a.part + n * a.chunks * a.C + c0;
    float s0 = 0.0f, s1 = 0.0f;
    for (int i = threadIdx.x % SPAN; i < items; i += SPAN) {
        const int k = i / a.D, c = i - k * a.D;
        const float w = a.w ? to_f32(static_cast<const T *>(a.w)[c0 + c]) : 1.0f;
        s0 = fmaf(w, m[(int64_t)k * a.C + c], s0);
        s1 = fmaf(w, m[half + (int64_t)k * a.C + c], s1);
    }
    s0 = span_sum<SPAN>(s0, s);
    s1 = span_sum<SPAN>(s1, s);
    const float total = (float)a.P * a.D;
    if (threadIdx.x % SPAN == 0) reinterpret_cast<float2 *>(a.sums)[id] = make_float2(s0 / total, s1 / total);
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS) gn_back_apply(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS, FEW = BATCH / 2;
    using Word = typename Group<T, V>::Word;
    const Place<T, V> at(a);
    tc::allow_dependents();
    tc::grid_dependency_wait();
    if (!at.in) return;
    const Channels<T, V> ch(a, at.n, at.c);
    F2 m1[PAIRS], m2[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        float v[2][2] = {};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (2 * i + j >= V) continue;
            const float2 s = reinterpret_cast<const float2 *>(a.sums)[at.n * a.G + (at.c + 2 * i + j) / a.D];
            v[0][j] = -s.x, v[1][j] = -s.y;
        }
        m1[i] = f2(v[0][0], v[0][1]), m2[i] = f2(v[1][0], v[1][1]);
    }
    with_norm_act(a.act, [&](auto kind) {
        for (int64_t p = at.p0 + at.row; p < at.p1; p += a.rows * FEW) {
            Word wx[FEW], wd[FEW];
#pragma unroll
            for (int j = 0; j < FEW; ++j)
                if (p + j * a.rows < at.p1) wx[j] = *at.at(a.x, a, p + j * a.rows), wd[j] = *at.at(a.dy, a, p + j * a.rows);
#pragma unroll
            for (int j = 0; j < FEW; ++j) {
                if (p + j * a.rows >= at.p1) continue;
                F2 x[PAIRS], d[PAIRS];
                to_pairs<T, V>(wx[j], x);
                to_pairs<T, V>(wd[j], d);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    const F2 hat = ch.hat(i, x[i]);
                    const F2 dz = mul2(d[i], slope_of<T, decltype(kind)::value>(fma2(hat, ch.w[i], ch.b[i])));
                    d[i] = mul2(fma2(hat, m2[i], fma2(dz, ch.w[i], m1[i])), ch.inv[i]);
                }
                *at.at(a.dx, a, p + j * a.rows) = from_pairs<T, V>(d);
            }
        }
    });
}

// dw and db: the channels' sums over images and chunks; 32 channels by 8 runs of rows a block.
template <typename T>
__global__ void __launch_bounds__(THREADS) gn_back_params(const __grid_constant__ GroupArgs a) {
    __shared__ float red[2][8][33];
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const int64_t rows = a.N * a.chunks, half = rows * a.C;
    float s0 = 0.0f, s1 = 0.0f;
    if (c < a.C) {
#pragma unroll 4
        for (int64_t r = run; r < rows; r += 8) s0 += a.part[r * a.C + c], s1 += a.part[half + r * a.C + c];
    }
    red[0][run][lane] = s0, red[1][run][lane] = s1;
    __syncthreads();
    if (run >= 2 || c >= a.C) return;
    T *out = static_cast<T *>(run ? a.dw : a.db);
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[run][i][lane];
    if (out) out[c] = from_f32<T>(t);
}

template <typename K>
cudaError_t launch(K kernel, int64_t blocks, cudaStream_t st, const GroupArgs &a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// A block a group where a warp would take more than 32 loads of each sum.
inline bool by_block(const GroupArgs &a) { return (int64_t)a.D * a.chunks > 1024; }
inline int64_t group_blocks(const GroupArgs &a) { return by_block(a) ? a.N * a.G : (a.N * a.G + 7) / 8; }

template <typename T, typename Fn>
cudaError_t with_vector(const GroupArgs &a, Fn f) {
    switch (vector_of(a.C, sizeof(T))) {
        case 1: return f(IntC<1>());
        case 2: return f(IntC<2>());
        default: return f(IntC<16 / (int)sizeof(T)>());
    }
}

}  // namespace

template <typename T>
cudaError_t launch_forward(const GroupArgs &a, cudaStream_t st) {
    const int64_t blocks = a.N * a.slabs * a.chunks;
    return with_vector<T>(a, [&](auto v) {
        constexpr int V = decltype(v)::value;
        cudaError_t e = launch(gn_moments<T, V>, blocks, st, a);
        if (e == cudaSuccess) e = by_block(a) ? launch(gn_stats<THREADS>, group_blocks(a), st, a) : launch(gn_stats<32>, group_blocks(a), st, a);
        return e == cudaSuccess ? launch(gn_apply<T, V>, blocks, st, a) : e;
    });
}

template <typename T>
cudaError_t launch_backward(const GroupArgs &a, cudaStream_t st) {
    const int64_t blocks = a.N * a.slabs * a.chunks;
    return with_vector<T>(a, [&](auto v) {
        constexpr int V = decltype(v)::value;
        cudaError_t e = launch(gn_back_sums<T, V>, blocks, st, a);
        if (a.dx) {
            if (e == cudaSuccess)
                e = by_block(a) ? launch(gn_back_means<T, THREADS>, group_blocks(a), st, a) : launch(gn_back_means<T, 32>, group_blocks(a), st, a);
            if (e == cudaSuccess) e = launch(gn_back_apply<T, V>, blocks, st, a);
        }
        if (e == cudaSuccess && (a.dw || a.db)) e = launch(gn_back_params<T>, (a.C + 31) / 32, st, a);
        return e;
    });
}

}  // namespace gnorm
}  // namespace im2win
