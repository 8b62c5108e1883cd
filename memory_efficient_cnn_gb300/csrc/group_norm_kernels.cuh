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
//
// Maps of up to 16 MB stay on the chip (one launch: 1 x 7 x 7 x 512 in 5 us, 13 x 31 x 37 x 90 of fp32 in 13 us forward
// and 16 us backward); larger ones are read twice. 64 x 56 x 56 x 128 of 16 bits: 12 us for the moments (51 MB, 4.2 TB/s),
// 3 for the statistics, 13 for the outputs; backward 23 for the sums (103 MB), 3 for the means, 24 for dx. Between a
// launch's first loads and its last sum over a block's rows 3 to 5 us go by that no other block fills; besides, half of
// the issue slots are taken.
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
// 1 / (1 + 2^a), two values with one reciprocal: 1/p and 1/q are q and p over pq. Half the
// instructions of the slowest unit: with a reciprocal each, silu over 51 million values took
// 25 us of the reading and writing pass's 31 us. (a is bounded so that pq stays finite; a NaN becomes a
// number here, which its neighbour needs: callers multiply by the value
// itself. Where a is bounded silu is z 2^-63, nothing next to z's rounding.)
__device__ __forceinline__ F2 logistic2(F2 a) {
    const F2 e = add2(exp2_2(each2(a, [](float v) { return fminf(v, 63.0f); })), f2(1.0f));
    float p, q, inv;
    split(e, p, q);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(p * q));
    return f2(inv * q, inv * p);
}
// act(z); fp32 by the functions themselves, 16-bit types by the approximations made for them.
template <typename T, int ACT>
__device__ __forceinline__ F2 act_of(F2 z) {
    if constexpr (ACT == IM2WIN_ACT_NONE) return z;
    else if constexpr (sizeof(T) == 4) return each2(z, [](float v) { return act_value<ACT>(v); });
    else if constexpr (ACT == IM2WIN_ACT_SILU) return mul2(z, logistic2(mul2(z, f2(-1.4426950408889634f))));
    else if constexpr (ACT == IM2WIN_ACT_GELU_TANH)  // -log2(e) 2 sqrt(2 / pi) (z + 0.044715 z^3)
        return mul2(z, logistic2(mul2(z, fma2(mul2(z, z), f2(-0.10294324f), f2(-2.3022082f)))));
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
    } else if constexpr (ACT == IM2WIN_ACT_SILU) {  // p + z p (1 - p)
        const F2 p = logistic2(mul2(z, f2(-1.4426950408889634f)));
        return fma2(mul2(z, p), fma2(p, f2(-1.0f), f2(1.0f)), p);
    } else if constexpr (ACT == IM2WIN_ACT_GELU_TANH) {  // p + z p (1 - p) a'(z); (the square is bounded: 0 times it stays 0)
        const F2 sq = each2(mul2(z, z), [](float v) { return v > 1e38f ? 1e38f : v; });
        const F2 p = logistic2(mul2(z, fma2(sq, f2(-0.10294324f), f2(-2.3022082f))));
        const F2 s = mul2(mul2(z, p), fma2(p, f2(-1.0f), f2(1.0f)));
        return fma2(s, fma2(sq, f2(0.21406859f), f2(1.5957691f)), p);
    } else {
        F2 a, d;
        act_both2<ACT>(z, a, d);
        return d;
    }
}
__device__ __forceinline__ F2 neg2(F2 a) { return mul2(a, f2(-1.0f)); }

// What a thread of the position passes works on: `count` positions, `step` elements apart.
template <typename T, int V>
struct Place {
    using Word = typename Group<T, V>::Word;
    int64_t n, first, step;  // image, first element
    int chunk, row, col, c, positions, count;  // c: first channel of the thread's vector; positions: of the block
    bool in;
    // last: in the opposite order, so that a second pass begins with what the first one has left in L2
    __device__ Place(const GroupArgs &a, bool last = false) {
        int64_t id = last ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
        chunk = (int)(id % a.chunks);
        id /= a.chunks;
        const int slab = (int)(id % a.slabs);
        n = id / a.slabs;
        row = threadIdx.x / a.cols, col = threadIdx.x - row * a.cols;
        c = (slab * a.cols + col) * V;
        in = row < a.rows && c < a.C;
        const int64_t p0 = chunk * a.len;
        positions = (int)(min(a.P, p0 + a.len) - p0);
        count = in ? count_of(a, row) : 0;
        first = (n * a.P + p0 + row) * a.C + c;
        step = (int64_t)a.rows * a.C;
    }
    __device__ int count_of(const GroupArgs &a, int r) const { return r < positions ? (positions - r + a.rows - 1) / a.rows : 0; }
    __device__ const T *at(const void *x) const { return static_cast<const T *>(x) + first; }
    __device__ T *at(void *x) const { return static_cast<T *>(x) + first; }
};
// A copy of this thread's, on its way to shared memory.
template <typename Word>
__device__ __forceinline__ void copy_ahead(Word *to, const void *from) {
    if constexpr (sizeof(Word) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
    else if constexpr (sizeof(Word) >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(to)), "l"(from), "n"(sizeof(Word)) : "memory");
    else
        *to = *static_cast<const Word *>(from);
}

// The vectors of a thread's positions, of MAPS tensors, through its own slots of shared memory: DEPTH - 1
// positions are under way while one is worked on, without registers for them (with the next vectors in
// registers the backward kernels had 16 warps an SM and read at half of the memory's rate).
template <int MAPS>
constexpr int RING_DEPTH = 8 / MAPS;
template <typename T, int V>
constexpr int RING_BYTES = 8 * THREADS * V * (int)sizeof(T);
// begin(slots) is called with the first DEPTH - 1 positions under way, f(position, vectors) for each of them.
template <typename T, int V, int MAPS, typename Begin, typename Fn>
__device__ __forceinline__ void each_vector(const Place<T, V> &at, const T *const (&src)[MAPS], void *ring, Begin begin, Fn f) {
    using Word = typename Group<T, V>::Word;
    constexpr int DEPTH = RING_DEPTH<MAPS>;
    Word *slots = static_cast<Word *>(ring) + threadIdx.x;
    const T *from[MAPS];
#pragma unroll
    for (int m = 0; m < MAPS; ++m) from[m] = src[m];
    int ahead = 0, put = 0, get = 0;
    auto start = [&] {
        if (ahead < at.count) {
#pragma unroll
            for (int m = 0; m < MAPS; ++m) {
                copy_ahead(slots + (put * MAPS + m) * THREADS, from[m]);
                from[m] += at.step;
            }
        }
        ++ahead;
        if (++put == DEPTH) put = 0;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) start();
    begin(slots);
#pragma unroll 1
    for (int k = 0; k < at.count; ++k) {
        start();
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        Word w[MAPS];
#pragma unroll
        for (int m = 0; m < MAPS; ++m) w[m] = slots[(get * MAPS + m) * THREADS];
        if (++get == DEPTH) get = 0;
        f(k, w);
    }
}
template <typename T, int V, int MAPS, typename Fn>
__device__ __forceinline__ void each_vector(const Place<T, V> &at, const T *const (&src)[MAPS], void *ring, Fn f) {
    each_vector<T, V, MAPS>(at, src, ring, [](auto *) {}, f);
}

// What makes z of the thread's channels: z = (x - mean) scale + b, scale = w / deviation.
template <typename T, int V>
struct Channels {
    static constexpr int PAIRS = Group<T, V>::PAIRS;
    F2 minus_mean[PAIRS], scale[PAIRS], b[PAIRS];
    __device__ Channels() {}
    __device__ Channels(const GroupArgs &a, int64_t n, int c) { load(a, n, c); }
    __device__ void load(const GroupArgs &a, int64_t n, int c) {
        each(a, n, c, [&](int i, const float2 (&s)[2], const float (&w)[2], const float (&bias)[2]) {
            minus_mean[i] = f2(-s[0].x, -s[1].x);
            scale[i] = f2(s[0].y * w[0], s[1].y * w[1]);
            b[i] = f2(bias[0], bias[1]);
        });
    }
    __device__ F2 z(int i, F2 deviation) const { return fma2(deviation, scale[i], b[i]); }
    // f(pair, its channels' mean and inverse deviation, w, b)
    template <typename Fn>
    static __device__ void each(const GroupArgs &a, int64_t n, int c, Fn f) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float2 s[2] = {};
            float w[2] = {}, b[2] = {};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (2 * i + j >= V) continue;
                const int ch = c + 2 * i + j;
                s[j] = reinterpret_cast<const float2 *>(a.stats)[n * a.G + ch / a.D];
                w[j] = a.w ? to_f32(static_cast<const T *>(a.w)[ch]) : 1.0f;
                b[j] = a.b ? to_f32(static_cast<const T *>(a.b)[ch]) : 0.0f;
            }
            f(i, s, w, b);
        }
    }
};

// dz of a vector and its deviations from the mean.
template <typename T, int V, int ACT>
__device__ __forceinline__ void gradients(const Channels<T, V> &ch, const typename Group<T, V>::Word &wx,
                                          const typename Group<T, V>::Word &wd, F2 (&dev)[Group<T, V>::PAIRS],
                                          F2 (&dz)[Group<T, V>::PAIRS]) {
    to_pairs<T, V>(wx, dev);
    to_pairs<T, V>(wd, dz);
#pragma unroll
    for (int i = 0; i < Group<T, V>::PAIRS; ++i) {
        dev[i] = add2(dev[i], ch.minus_mean[i]);
        dz[i] = mul2(dz[i], slope_of<T, ACT>(ch.z(i, dev[i])));
    }
}
// dx of them: i w dz - i (m1 + hat m2), with the group's means m1 of w dz and m2 of w dz hat.
template <typename T, int V>
struct Back {
    static constexpr int PAIRS = Group<T, V>::PAIRS;
    F2 base[PAIRS], slope[PAIRS];  // - i m1, - i^2 m2
    // of(group): its -m1 and -m2; c: the first channel
    template <typename Fn>
    __device__ void load(const GroupArgs &a, int64_t n, int c, Fn of) {
        Channels<T, V>::each(a, n, c, [&](int i, const float2 (&s)[2], const float (&)[2], const float (&)[2]) {
            float2 m[2] = {};
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (2 * i + j < V) m[j] = of((c + 2 * i + j) / a.D);
            base[i] = f2(m[0].x * s[0].y, m[1].x * s[1].y);
            slope[i] = f2(m[0].y * s[0].y * s[0].y, m[1].y * s[1].y * s[1].y);
        });
    }
    __device__ F2 dx(const Channels<T, V> &ch, int i, F2 dev, F2 dz) const {
        return fma2(dev, slope[i], fma2(dz, ch.scale[i], base[i]));
    }
};

// A thread's channels' two sums, row `row` of the partial ones.
template <int V, int PAIRS>
__device__ __forceinline__ void store_channels(const GroupArgs &a, int64_t row, int c, const F2 (&v)[PAIRS], const F2 (&u)[PAIRS]) {
    float *m = a.part + row * a.C + c, *q = m + a.part_rows * a.C;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        float lo, hi, lo2, hi2;
        split(v[i], lo, hi);
        split(u[i], lo2, hi2);
        m[2 * i] = lo, q[2 * i] = lo2;
        if (V > 1) m[2 * i + 1] = hi, q[2 * i + 1] = hi2;
    }
}

// Means and sums of squared deviations of a chunk's positions, for each channel. A thread sums deviations from the
// mean of its first positions; what the sum of squares loses to a pivot that is d from its mean is 2^-24 n d^2 of its n
// values, of which an outlier among the FIRST makes at most n / FIRST^2 of its own square.
template <typename T, int V>
__global__ void __launch_bounds__(THREADS, 4) gn_moments(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS, FIRST = 4;
    using Word = typename Group<T, V>::Word;
    __shared__ alignas(16) unsigned char ring[std::max(RING_BYTES<T, V>, 2 * PAIRS * THREADS * 8)];
    __shared__ float counts[THREADS];
    F2(*red)[THREADS] = reinterpret_cast<F2(*)[THREADS]>(ring);
    const Place<T, V> at(a);
    // (in this order: the last launch of a call reads its inputs ahead of its own wait)
    tc::grid_dependency_wait();
    tc::allow_dependents();
    F2 mean[PAIRS], m2[PAIRS], pivot[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) mean[i] = m2[i] = pivot[i] = f2(0.0f);
    const T *const src[1] = {at.at(a.x)};
    auto take_pivot = [&](const Word *slots) {
        asm volatile("cp.async.wait_group %0;" ::"n"(RING_DEPTH<1> - 1 - FIRST) : "memory");
        const F2 share = f2(-1.0f / (float)max(1, min(FIRST, at.count)));  // (the negative pivot)
#pragma unroll
        for (int j = 0; j < FIRST; ++j) {
            if (j >= at.count) continue;
            F2 v[PAIRS];
            to_pairs<T, V>(slots[j * THREADS], v);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) pivot[i] = add2(pivot[i], v[i]);
        }
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) pivot[i] = mul2(pivot[i], share);
    };
    each_vector<T, V, 1>(at, src, ring, take_pivot, [&](int, const Word (&w)[1]) {
        F2 v[PAIRS];
        to_pairs<T, V>(w[0], v);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const F2 d = add2(v[i], pivot[i]);
            mean[i] = add2(mean[i], d);
            m2[i] = fma2(d, d, m2[i]);
        }
    });
    __syncthreads();  // (the ring becomes `red`)
    float count = (float)at.count;
    if (at.count > 0) {
        const F2 share = f2(1.0f / count);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const F2 d = mul2(mean[i], share);
            m2[i] = each2(fma2(mul2(d, mean[i]), f2(-1.0f), m2[i]), [](float v) { return v < 0.0f ? 0.0f : v; });
            mean[i] = add2(d, neg2(pivot[i]));
        }
    }
    // over the block's rows, in halves
    if (at.col == 0 && at.row < a.rows) counts[at.row] = (float)at.count_of(a, at.row);
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
            const float total = count + other, share = other / total, scale = count * share;
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const F2 d = add2(red[2 * i][t], neg2(mean[i]));
                mean[i] = fma2(d, f2(share), mean[i]);
                m2[i] = fma2(mul2(d, d), f2(scale), add2(m2[i], red[2 * i + 1][t]));
            }
            count = total;
        }
        __syncthreads();
        if (at.col == 0 && at.row < n - h) counts[at.row] += other;
        n = h;
        __syncthreads();
    }
    if (at.in && at.row == 0) store_channels<V>(a, at.n * a.chunks + at.chunk, at.c, mean, m2);
}

// Sum over SPAN threads (part of a warp, a warp, or the block), the same for each and in a fixed order.
template <int SPAN>
__device__ __forceinline__ float span_sum(float v, float *s) {
#pragma unroll
    for (int o = (SPAN < 32 ? SPAN : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (SPAN <= 32) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < SPAN / 32; ++i) t += s[i];
    __syncthreads();
    return t;
}

// The sums of two values at once.
template <int SPAN>
__device__ __forceinline__ float2 span_sums(float2 v, float2 *s) {
    v = make_float2(span_sum<SPAN < 32 ? SPAN : 32>(v.x, nullptr), span_sum<SPAN < 32 ? SPAN : 32>(v.y, nullptr));
    if (SPAN <= 32) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < SPAN / 32; ++i) v.x += s[i].x, v.y += s[i].y;
    return v;
}

// A group's chunks and channels become its mean and inverse deviation; SPAN threads a group. Twice over them: the
// deviations are those from the group's own mean, and their sum is what the first pass's rounding left of it. (From a
// pivot, sum of squares less square of the sum: a first chunk a hundred deviations away took 2e-3 of the variance
// of 36000 items.)
template <int SPAN>
__global__ void __launch_bounds__(THREADS) gn_stats(const __grid_constant__ GroupArgs a) {
    __shared__ float s[THREADS / 32];
    __shared__ float2 s2[THREADS / 32];
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t wanted = (int64_t)blockIdx.x * (THREADS / SPAN) + threadIdx.x / SPAN;
    const int64_t id = min(wanted, a.N * a.G - 1);  // (every lane takes part in the exchanges)
    const int64_t n = id / a.G, half = a.part_rows * a.C;
    const int c0 = (int)(id % a.G) * a.D, items = a.D * a.chunks;
    const float *m = a.part + n * a.chunks * a.C + c0;
    const float total = (float)a.P * a.D, share = 1.0f / total;
    // an item's place, and its number of positions
    auto item = [&](int i, int64_t &at) {
        const int k = i / a.D;
        at = (int64_t)k * a.C + i - k * a.D;
        return (float)(min(a.P, (k + 1) * a.len) - k * a.len);
    };
    // a thread's first items stay in registers (all of a group, but for a block's)
    constexpr int KEEP = 8;
    const int t = threadIdx.x % SPAN;
    float means[KEEP], squares[KEEP], counts[KEEP];
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        means[j] = squares[j] = counts[j] = 0.0f;
        if (t + j * SPAN >= items) continue;
        int64_t at;
        counts[j] = item(t + j * SPAN, at);
        means[j] = m[at], squares[j] = m[half + at];
    }
    float mean = 0.0f, sum = 0.0f, sq = 0.0f;
#pragma unroll
    for (int j = 0; j < KEEP; ++j) mean = fmaf(means[j], counts[j] * share, mean);
#pragma unroll 4
    for (int i = t + KEEP * SPAN; i < items; i += SPAN) {
        int64_t at;
        const float count = item(i, at);
        mean = fmaf(m[at], count * share, mean);
    }
    mean = span_sum<SPAN>(mean, s);
    auto add = [&](float d, float count, float square) {
        sum = fmaf(d, count, sum);
        sq += fmaf(d * count, d, square);
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
        if (t + j * SPAN < items) add(means[j] - mean, counts[j], squares[j]);
#pragma unroll 4
    for (int i = t + KEEP * SPAN; i < items; i += SPAN) {
        int64_t at;
        const float count = item(i, at);
        add(m[at] - mean, count, m[half + at]);
    }
    const float2 both = span_sums<SPAN>(make_float2(sum, sq), s2);
    sum = both.x, sq = both.y - sum * share * sum;
    if (t == 0 && wanted == id)
        reinterpret_cast<float2 *>(a.stats)[id] = make_float2(mean + sum * share, 1.0f / sqrtf((sq < 0.0f ? 0.0f : sq) * share + a.eps));
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS, 4) gn_apply(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    __shared__ alignas(16) unsigned char ring[RING_BYTES<T, V>];
    const Place<T, V> at(a, true);
    tc::allow_dependents();
    const T *const src[1] = {at.at(a.x)};
    T *y = at.at(a.y);
    Channels<T, V> ch;
    // x on its way before the statistics are there
    auto begin = [&](const Word *) {
        tc::grid_dependency_wait();
        if (at.in) ch.load(a, at.n, at.c);
    };
    with_norm_act(a.act, [&](auto kind) {
        each_vector<T, V, 1>(at, src, ring, begin, [&](int k, const Word (&w)[1]) {
            F2 v[PAIRS];
            to_pairs<T, V>(w[0], v);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) v[i] = act_of<T, decltype(kind)::value>(ch.z(i, add2(v[i], ch.minus_mean[i])));
            __stcs(reinterpret_cast<Word *>(y + k * at.step), from_pairs<T, V>(v));
        });
    });
}

// Sums of dz and dz xh over a chunk's positions, for each channel.
template <typename T, int V>
__global__ void __launch_bounds__(THREADS, 3) gn_back_sums(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    __shared__ alignas(16) unsigned char ring[std::max(RING_BYTES<T, V>, 2 * PAIRS * THREADS * 8)];
    F2(*red)[THREADS] = reinterpret_cast<F2(*)[THREADS]>(ring);
    const Place<T, V> at(a);
    // (in this order: the last launch of a call reads its inputs ahead of its own wait)
    tc::grid_dependency_wait();
    tc::allow_dependents();
    F2 s0[PAIRS], s1[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) s0[i] = s1[i] = f2(0.0f);
    if (at.in) {
        const Channels<T, V> ch(a, at.n, at.c);
        const T *const src[2] = {at.at(a.x), at.at(a.dy)};
        with_norm_act(a.act, [&](auto kind) {
            each_vector<T, V, 2>(at, src, ring, [&](int, const Word (&w)[2]) {
                F2 dev[PAIRS], dz[PAIRS];
                gradients<T, V, decltype(kind)::value>(ch, w[0], w[1], dev, dz);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    s0[i] = add2(s0[i], dz[i]);
                    s1[i] = fma2(dz[i], dev[i], s1[i]);
                }
            });
        });
        Channels<T, V>::each(a, at.n, at.c, [&](int i, const float2 (&s)[2], const float (&)[2], const float (&)[2]) {
            s1[i] = mul2(s1[i], f2(s[0].y, s[1].y));  // deviations to normed values
        });
    }
    __syncthreads();  // (the ring becomes `red`)
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
    if (at.in && at.row == 0) store_channels<V>(a, at.n * a.chunks + at.chunk, at.c, s0, s1);
}

// A group's means of w dz and w dz xh; SPAN threads a group.
template <typename T, int SPAN>
__global__ void __launch_bounds__(THREADS) gn_back_means(const __grid_constant__ GroupArgs a) {
    __shared__ float s[THREADS / 32];
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t id = (int64_t)blockIdx.x * (THREADS / SPAN) + threadIdx.x / SPAN;
    if (id >= a.N * a.G) return;
    const int64_t n = id / a.G, half = a.part_rows * a.C;
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

// The sums of rows `begin` to `end` of both halves of `part` (each of `rows` rows), for 32 channels: put(half, channel, sum).
template <typename Fn>
__device__ __forceinline__ void sum_rows(const GroupArgs &a, const float *part, int64_t rows, int64_t begin, int64_t end, int block, Fn put) {
    __shared__ float red[2][8][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c = block * 32 + lane;
    const int64_t half = rows * a.C;
    float s0 = 0.0f, s1 = 0.0f;
    if (c < a.C) {
#pragma unroll 8
        for (int64_t r = begin + run; r < end; r += 8) s0 += part[r * a.C + c], s1 += part[half + r * a.C + c];
    }
    red[0][run][lane] = s0, red[1][run][lane] = s1;
    __syncthreads();
    if (run >= 2 || c >= a.C) return;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[run][i][lane];
    put(run, c, t);
}
// dw and db: the channels' sums over images and chunks, or over the runs of those.
template <typename T>
__device__ __forceinline__ void sum_params(const GroupArgs &a, int block) {
    const int64_t rows = a.folds ? a.folds : a.part_rows;
    sum_rows(a, a.folds ? a.folded : a.part, rows, 0, rows, block, [&](int half, int c, float sum) {
        T *out = static_cast<T *>(half ? a.dw : a.db);
        if (out) out[c] = from_f32<T>(sum);
    });
}
template <typename T>
__global__ void __launch_bounds__(THREADS) gn_back_params(const __grid_constant__ GroupArgs a) {
    tc::allow_dependents();
    tc::grid_dependency_wait();
    sum_params<T>(a, blockIdx.x);
}
// The partial sums in a.folds runs of rows, a block for a run's 32 channels.
__global__ void __launch_bounds__(THREADS) gn_back_fold(const __grid_constant__ GroupArgs a) {
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t f = blockIdx.x % a.folds, per = (a.part_rows + a.folds - 1) / a.folds;
    sum_rows(a, a.part, a.part_rows, f * per, min(a.part_rows, (f + 1) * per), blockIdx.x / a.folds,
             [&](int half, int c, float sum) { a.folded[(half * (int64_t)a.folds + f) * a.C + c] = sum; });
}

// dx; the first `param_blocks` blocks make dw and db meanwhile.
template <typename T, int V>
__global__ void __launch_bounds__(THREADS, 3) gn_back_apply(const __grid_constant__ GroupArgs a, int param_blocks) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    __shared__ alignas(16) unsigned char ring[RING_BYTES<T, V>];
    tc::allow_dependents();
    if ((int)blockIdx.x < param_blocks) {
        tc::grid_dependency_wait();
        sum_params<T>(a, blockIdx.x);
        return;
    }
    const Place<T, V> at(a, true);
    Channels<T, V> ch;
    Back<T, V> back;
    auto begin = [&](const Word *) {  // (as above)
        tc::grid_dependency_wait();
        if (!at.in) return;
        ch.load(a, at.n, at.c);
        back.load(a, at.n, at.c, [&](int g) {
            const float2 s = reinterpret_cast<const float2 *>(a.sums)[at.n * a.G + g];
            return make_float2(-s.x, -s.y);
        });
    };
    T *dx = at.at(a.dx);
    const T *const src[2] = {at.at(a.x), at.at(a.dy)};
    with_norm_act(a.act, [&](auto kind) {
        each_vector<T, V, 2>(at, src, ring, begin, [&](int k, const Word (&w)[2]) {
            F2 dev[PAIRS], dz[PAIRS];
            gradients<T, V, decltype(kind)::value>(ch, w[0], w[1], dev, dz);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) dz[i] = back.dx(ch, i, dev[i], dz[i]);
            __stcs(reinterpret_cast<Word *>(dx + k * at.step), from_pairs<T, V>(dz));
        });
    });
}

// ---- resident: an image's slab of channels stays in shared memory between the passes over it

// What a CTA of a cluster works on: positions p0 to p1 of image n, channels c0 to c0 + sc. A thread keeps to
// one vector of channels and takes every rows-th position; its i-th vector lies at tile[i * THREADS + tid].
template <typename T, int V>
struct Seat {
    using Word = typename Group<T, V>::Word;
    int64_t n, p0, p1, base;
    int rank, c0, sc, cols, rows, row, col, c;
    bool in;
    __device__ explicit Seat(const GroupArgs &a) {
        rank = blockIdx.x % a.chunks;
        const int64_t id = blockIdx.x / a.chunks;
        n = id / a.slabs;
        c0 = (int)(id - n * a.slabs) * a.slab;
        sc = min(a.slab, a.C - c0);
        cols = sc / V, rows = THREADS / cols;
        row = threadIdx.x / cols, col = threadIdx.x - row * cols;
        in = row < rows;
        c = c0 + col * V;
        p0 = min(a.P, rank * a.len), p1 = min(a.P, p0 + a.len);
        base = n * a.P * a.C + c;
    }
    // the thread's vectors of x on their way to the tile
    __device__ void fetch(const GroupArgs &a, const void *x, Word *tile) const {
        if (!in) return;
        const T *from = static_cast<const T *>(x) + base + (p0 + row) * a.C;
        const int64_t step = (int64_t)rows * a.C;
        Word *to = tile + threadIdx.x;
        for (int64_t p = p0 + row; p < p1; p += rows, from += step, to += THREADS) copy_ahead(to, from);
    }
    // f(i-th vector's pairs, position) for each of the thread's vectors
    template <typename Fn>
    __device__ void each(Fn f) const {
        if (!in) return;
        int at = threadIdx.x;
        for (int64_t p = p0 + row; p < p1; p += rows, at += THREADS) f(at, p);
    }
};
__device__ __forceinline__ void wait_fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Scratch of the sums over a CTA.
struct Sums {
    float *each, *channel, *group;  // [SUMS][THREADS * V], [SUMS][segments * sc], [SUMS][groups]
    int segments;
};
// The sums of SUMS values over the CTA's positions, by channel (in `segments` parts) and, `weight` times them,
// by group. Every thread calls this; the results may be read after it.
template <typename T, int V, int SUMS, typename Fn>
__device__ __forceinline__ void sum_groups(const GroupArgs &a, const Seat<T, V> &at, Sums &s,
                                           const F2 (&v)[SUMS][Group<T, V>::PAIRS], Fn weight) {
    constexpr int EACH = THREADS * V;
    const int wide = max(THREADS, at.sc), groups = at.sc / a.D;
    if (at.in) {
#pragma unroll
        for (int q = 0; q < SUMS; ++q)
#pragma unroll
            for (int i = 0; i < Group<T, V>::PAIRS; ++i) {
                float lo, hi;
                split(v[q][i], lo, hi);
                s.each[q * EACH + threadIdx.x * V + 2 * i] = lo;
                if (V > 1) s.each[q * EACH + threadIdx.x * V + 2 * i + 1] = hi;
            }
    }
    __syncthreads();
    s.segments = max(1, THREADS / at.sc);
    const int per = (at.rows + s.segments - 1) / s.segments;
    for (int id = threadIdx.x; id < s.segments * at.sc; id += THREADS) {
        const int seg = id / at.sc, c = id - seg * at.sc;
        float sum[SUMS] = {};
        for (int r = seg * per; r < min(at.rows, (seg + 1) * per); ++r)
#pragma unroll
            for (int q = 0; q < SUMS; ++q) sum[q] += s.each[q * EACH + r * at.sc + c];
#pragma unroll
        for (int q = 0; q < SUMS; ++q) s.channel[q * wide + id] = sum[q];
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < groups; g += THREADS / 32) {
        float sum[SUMS] = {};
        for (int j = lane; j < s.segments * a.D; j += 32) {
            const int seg = j / a.D, c = g * a.D + j - seg * a.D;
            const float w = weight(c);
#pragma unroll
            for (int q = 0; q < SUMS; ++q) sum[q] = fmaf(w, s.channel[q * wide + seg * at.sc + c], sum[q]);
        }
#pragma unroll
        for (int q = 0; q < SUMS; ++q) {
            sum[q] = span_sum<32>(sum[q], nullptr);
            if (lane == 0) s.group[q * groups + g] = sum[q];
        }
    }
    __syncthreads();
}
__device__ __forceinline__ float peer_read(const float *p, int rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The parts of a resident CTA's shared memory behind its tiles.
template <typename T, int V, int SUMS>
__device__ __forceinline__ Sums scratch(const GroupArgs &a, int sc, unsigned char *at) {
    float *p = reinterpret_cast<float *>(at);
    return {p, p + SUMS * THREADS * V, p + SUMS * (THREADS * V + max(THREADS, sc)), 0};
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS) gn_resident(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    extern __shared__ uint4 dyn[];
    const Seat<T, V> at(a);
    Word *tile = reinterpret_cast<Word *>(dyn);
    Sums s = scratch<T, V, 2>(a, at.sc, reinterpret_cast<unsigned char *>(dyn) + a.tile);
    tc::allow_dependents();
    tc::grid_dependency_wait();
    at.fetch(a, a.x, tile);
    F2 w[PAIRS], b[PAIRS];
    int group[V];  // of the thread's channels, in the slab
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        float v[2][2] = {};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (2 * i + j >= V) continue;
            const int ch = min(at.c + 2 * i + j, a.C - 1);
            group[2 * i + j] = min(at.col * V + 2 * i + j, at.sc - 1) / a.D;
            v[0][j] = a.w ? to_f32(static_cast<const T *>(a.w)[ch]) : 1.0f;
            v[1][j] = a.b ? to_f32(static_cast<const T *>(a.b)[ch]) : 0.0f;
        }
        w[i] = f2(v[0][0], v[0][1]), b[i] = f2(v[1][0], v[1][1]);
    }
    auto of_groups = [&](const float *of, F2 (&v)[PAIRS]) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) v[i] = f2(of[group[2 * i]], V > 1 ? of[group[V > 1 ? 2 * i + 1 : 0]] : 0.0f);
    };
    wait_fetched();
    const int groups = at.sc / a.D;
    constexpr int SUMS = sizeof(T) == 4 ? 2 : 1;
    F2 total[1][PAIRS], sum[SUMS][PAIRS], mean[PAIRS], inv[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) total[0][i] = sum[0][i] = sum[SUMS - 1][i] = f2(0.0f);
    at.each([&](int j, int64_t) {
        F2 v[PAIRS];
        to_pairs<T, V>(tile[j], v);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) total[0][i] = add2(total[0][i], v[i]);
    });
    sum_groups<T, V, 1>(a, at, s, total, [](int) { return 1.0f; });
    // the CTA's own mean and the squared deviations from it; fp32, also their sum: what the first sum's rounding left of the
    // mean. (16-bit values of a mean so far away that this counts hold fewer digits themselves, and it takes
    // 32768 images of 4 x 32 from 410 to 590 us.)
    float *means = s.group + groups, *m2 = s.group;
    const float count = (float)(at.p1 - at.p0) * a.D;
    float own = 0.0f;  // of group threadIdx.x (a slab has 64 at most)
    if (threadIdx.x < groups) means[threadIdx.x] = own = count > 0.0f ? s.group[threadIdx.x] / count : 0.0f;
    __syncthreads();
    of_groups(means, mean);
    at.each([&](int j, int64_t) {
        F2 v[PAIRS];
        to_pairs<T, V>(tile[j], v);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const F2 d = add2(v[i], neg2(mean[i]));
            sum[0][i] = fma2(d, d, sum[0][i]);
            if (SUMS == 2) sum[SUMS - 1][i] = add2(sum[SUMS - 1][i], d);
        }
    });
    sum_groups<T, V, SUMS>(a, at, s, sum, [](int) { return 1.0f; });
    if (SUMS == 2 && threadIdx.x < groups) {
        const float left = means[threadIdx.x], off = count > 0.0f ? left / count : 0.0f, q = m2[threadIdx.x] - off * left;
        means[threadIdx.x] = own + off;
        m2[threadIdx.x] = q < 0.0f ? 0.0f : q;
    }
    // the cluster's; results go where no other CTA reads
    if (a.chunks > 1) cluster_barrier();
    float *result = s.channel;  // [2][groups]
    for (int g = threadIdx.x; g < groups; g += THREADS) {
        float m = means[g], q = m2[g];
        if (a.chunks > 1) {
            // (all on their way before the first is used; the first CTA has positions wherever there are any)
            const int len = (int)a.len, left = (int)a.P;  // (below 2^24: the maps are)
            float mr[MOST_SHARES], qr[MOST_SHARES], nr[MOST_SHARES], total = 0.0f;
#pragma unroll
            for (int r = 0; r < MOST_SHARES; ++r) {
                mr[r] = r < a.chunks ? peer_read(means + g, r) : 0.0f;
                qr[r] = r < a.chunks ? peer_read(m2 + g, r) : 0.0f;
                nr[r] = (float)max(0, min(len, left - r * len));
            }
#pragma unroll
            for (int r = 0; r < MOST_SHARES; ++r) total = fmaf(mr[r] - mr[0], nr[r], total);
            m = mr[0] + total / (float)a.P;
            q = 0.0f;
#pragma unroll
            for (int r = 0; r < MOST_SHARES; ++r) q += fmaf((mr[r] - m) * (mr[r] - m), nr[r] * a.D, qr[r]);
        }
        const float i = 1.0f / sqrtf(q / ((float)a.P * a.D) + a.eps);
        result[g] = m, result[groups + g] = i;
        if (a.stats && at.rank == 0) reinterpret_cast<float2 *>(a.stats)[at.n * a.G + at.c0 / a.D + g] = make_float2(m, i);
    }
    // (the others' scratch is read no more after this: they may go on, or end)
    if (a.chunks > 1) cluster_barrier();
    else __syncthreads();
    of_groups(result, mean);
    of_groups(result + groups, inv);
    with_norm_act(a.act, [&](auto kind) {
        at.each([&](int j, int64_t p) {
            F2 v[PAIRS];
            to_pairs<T, V>(tile[j], v);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i)
                v[i] = act_of<T, decltype(kind)::value>(fma2(mul2(add2(v[i], neg2(mean[i])), inv[i]), w[i], b[i]));
            *reinterpret_cast<Word *>(static_cast<T *>(a.y) + at.base + p * a.C) = from_pairs<T, V>(v);
        });
    });
}

// Backward: x and dy in shared memory; the channels' sums go to `part` for dw and db.
template <typename T, int V>
__global__ void __launch_bounds__(THREADS) gn_back_resident(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    extern __shared__ uint4 dyn[];
    const Seat<T, V> at(a);
    Word *xs = reinterpret_cast<Word *>(dyn);
    Word *ds = reinterpret_cast<Word *>(reinterpret_cast<unsigned char *>(dyn) + a.tile / 2);
    Sums s = scratch<T, V, 2>(a, at.sc, reinterpret_cast<unsigned char *>(dyn) + a.tile);
    tc::allow_dependents();
    tc::grid_dependency_wait();
    at.fetch(a, a.x, xs);
    at.fetch(a, a.dy, ds);
    const Channels<T, V> ch(a, at.n, at.in ? at.c : at.c0);
    wait_fetched();
    F2 sum[2][PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) sum[0][i] = sum[1][i] = f2(0.0f);
    with_norm_act(a.act, [&](auto kind) {
        at.each([&](int j, int64_t) {
            F2 dev[PAIRS], dz[PAIRS];
            gradients<T, V, decltype(kind)::value>(ch, xs[j], ds[j], dev, dz);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                sum[0][i] = add2(sum[0][i], dz[i]);
                sum[1][i] = fma2(dz[i], dev[i], sum[1][i]);
            }
        });
    });
    Channels<T, V>::each(a, at.n, at.in ? at.c : at.c0, [&](int i, const float2 (&t)[2], const float (&)[2], const float (&)[2]) {
        sum[1][i] = mul2(sum[1][i], f2(t[0].y, t[1].y));  // deviations to normed values
    });
    sum_groups<T, V, 2>(a, at, s, sum, [&](int c) { return a.w ? to_f32(static_cast<const T *>(a.w)[at.c0 + c]) : 1.0f; });
    const int groups = at.sc / a.D, wide = max(THREADS, at.sc);
    if (a.dw || a.db) {
        const int64_t row = (at.n * a.chunks + at.rank) * a.C + at.c0, half = a.part_rows * a.C;
        for (int c = threadIdx.x; c < at.sc; c += THREADS) {
            float t[2] = {};
            for (int seg = 0; seg < s.segments; ++seg) t[0] += s.channel[seg * at.sc + c], t[1] += s.channel[wide + seg * at.sc + c];
            a.part[row + c] = t[0], a.part[half + row + c] = t[1];
        }
    }
    if (!a.dx) return;  // (of every CTA alike)
    if (a.chunks > 1) cluster_barrier();
    else __syncthreads();
    float *result = s.each;  // [2][groups]
    for (int g = threadIdx.x; g < groups; g += THREADS) {
        float t[2] = {s.group[g], s.group[groups + g]};
        if (a.chunks > 1) {
            float part[2][MOST_SHARES];
#pragma unroll
            for (int r = 0; r < MOST_SHARES; ++r)
#pragma unroll
                for (int q = 0; q < 2; ++q) part[q][r] = r < a.chunks ? peer_read(s.group + q * groups + g, r) : 0.0f;
            t[0] = t[1] = 0.0f;
#pragma unroll
            for (int r = 0; r < MOST_SHARES; ++r) t[0] += part[0][r], t[1] += part[1][r];
        }
        const float total = (float)a.P * a.D;
        result[g] = -t[0] / total, result[groups + g] = -t[1] / total;
    }
    if (a.chunks > 1) cluster_barrier();
    else __syncthreads();
    const int g0 = at.c0 / a.D;
    Back<T, V> back;
    back.load(a, at.n, at.in ? at.c : at.c0, [&](int g) { return make_float2(result[g - g0], result[groups + g - g0]); });
    with_norm_act(a.act, [&](auto kind) {
        at.each([&](int j, int64_t p) {
            F2 dev[PAIRS], dz[PAIRS];
            gradients<T, V, decltype(kind)::value>(ch, xs[j], ds[j], dev, dz);
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) dz[i] = back.dx(ch, i, dev[i], dz[i]);
            *reinterpret_cast<Word *>(static_cast<T *>(a.dx) + at.base + p * a.C) = from_pairs<T, V>(dz);
        });
    });
}

// ---- one position an image: a group is D neighbouring elements of a row, in the registers of a.lanes lanes; the next
// row's are on their way. 200704 rows of 512 channels in 8 groups, bf16 and silu: 108 us forward, 181 us backward (3.8
// and 3.4 TB/s), bound by instructions and the lanes' exchanges (79 and 68% of the issue slots).

// A thread's group and vectors: the m-th one begins at element d(m) of the group where it is there.
template <typename T, int V, int M>
struct RowSeat {
    using Word = typename Group<T, V>::Word;
    int row, lane, g, vecs, lanes;
    int64_t n, step;
    bool in;
    __device__ explicit RowSeat(const GroupArgs &a) {
        const int slab = blockIdx.x % a.slabs, slot = threadIdx.x % a.cols + slab * a.cols;
        row = threadIdx.x / a.cols;
        lanes = a.lanes, lane = slot % lanes, g = slot / lanes, vecs = a.D / V;
        in = row < a.rows && g < a.G;
        n = (int64_t)(blockIdx.x / a.slabs) * a.rows + row;
        step = (int64_t)a.chunks * a.rows;
    }
    __device__ bool has(int m) const { return lane + m * lanes < vecs; }
    __device__ int channel(const GroupArgs &a, int m) const { return g * a.D + (lane + m * lanes) * V; }
    __device__ float sum(float v) const {
        for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
};
// The sum of a pair's elements (V = 1: there is one).
template <int V>
__device__ __forceinline__ float pair_sum(F2 v) {
    float lo, hi;
    split(v, lo, hi);
    return V > 1 ? lo + hi : lo;
}
// A thread's vectors of a row (or of the parameters: n = 0) on their way.
template <typename T, int V, int M>
__device__ __forceinline__ void fetch_row(const GroupArgs &a, const RowSeat<T, V, M> &at, const void *p, int64_t n,
                                          typename Group<T, V>::Word (&w)[M]) {
    if (!p || !at.in || n >= a.N) return;
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (at.has(m))
            w[m] = *reinterpret_cast<const typename Group<T, V>::Word *>(static_cast<const T *>(p) + n * a.C + at.channel(a, m));
}
template <typename T, int V>
__device__ __forceinline__ void params_of(const void *p, const typename Group<T, V>::Word &word, float absent,
                                          F2 (&v)[Group<T, V>::PAIRS]) {
    if (p) {
        to_pairs<T, V>(word, v);
    } else {
#pragma unroll
        for (int i = 0; i < Group<T, V>::PAIRS; ++i) v[i] = f2(absent);
    }
}

template <typename T, int V, int M>
__global__ void __launch_bounds__(THREADS) gn_rows(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    const RowSeat<T, V, M> at(a);
    tc::grid_dependency_wait();
    tc::allow_dependents();
    const float share = 1.0f / (float)a.D;
    constexpr bool AHEAD = M <= 2;  // (four vectors take the registers themselves)
    Word ww[M], wb[M], next[M];
    if (AHEAD) fetch_row(a, at, a.x, at.n, next);
    fetch_row(a, at, a.w, 0, ww);
    fetch_row(a, at, a.b, 0, wb);
    with_norm_act(a.act, [&](auto kind) {
        for (int64_t n = at.n; n - at.row < a.N; n += at.step) {  // (as often for every row of the block: lanes exchange)
            const bool there = at.in && n < a.N;
            if (!AHEAD) fetch_row(a, at, a.x, n, next);
            Word word[M];
#pragma unroll
            for (int m = 0; m < M; ++m) word[m] = next[m];
            if (AHEAD) fetch_row(a, at, a.x, n + at.step, next);
            // fp32: the sum of distances to the group's first value, so that a far mean costs its own rounding alone
            // (and the first one of at most 1024 is 32 deviations from it at most). 16-bit values with a mean so far away hold
            // fewer digits than it costs; for them it took 116 us instead of 111 us.
            F2 v[M][PAIRS];
            float s = 0.0f, pivot = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) v[m][i] = f2(0.0f);
                if (there && at.has(m)) to_pairs<T, V>(word[m], v[m]);
                if (sizeof(T) == 4 && m == 0) {
                    float unused;
                    split(v[0][0], pivot, unused);
                    pivot = __shfl_sync(0xffffffffu, pivot, threadIdx.x & 31 & ~(at.lanes - 1));
                }
                if (sizeof(T) == 4 && !at.has(m)) continue;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    if (sizeof(T) == 4) v[m][i] = add2(v[m][i], f2(-pivot));
                    s += pair_sum<V>(v[m][i]);
                }
            }
            const float off = at.sum(s) * share, mean = pivot + off;
            s = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (!at.has(m)) continue;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    v[m][i] = add2(v[m][i], f2(-off));
                    s += pair_sum<V>(mul2(v[m][i], v[m][i]));
                }
            }
            const float inv = 1.0f / sqrtf(at.sum(s) * share + a.eps);
            if (!there) continue;
            if (a.stats && at.lane == 0) reinterpret_cast<float2 *>(a.stats)[n * a.G + at.g] = make_float2(mean, inv);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (!at.has(m)) continue;
                F2 w[PAIRS], b[PAIRS];
                params_of<T, V>(a.w, ww[m], 1.0f, w);
                params_of<T, V>(a.b, wb[m], 0.0f, b);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i)
                    v[m][i] = act_of<T, decltype(kind)::value>(fma2(v[m][i], mul2(w[i], f2(inv)), b[i]));
                *reinterpret_cast<Word *>(static_cast<T *>(a.y) + n * a.C + at.channel(a, m)) = from_pairs<T, V>(v[m]);
            }
        }
    });
}

template <typename T, int V, int M>
__global__ void __launch_bounds__(THREADS) gn_back_rows(const __grid_constant__ GroupArgs a) {
    constexpr int PAIRS = Group<T, V>::PAIRS;
    using Word = typename Group<T, V>::Word;
    __shared__ F2 red[2 * PAIRS][THREADS];
    const RowSeat<T, V, M> at(a);
    tc::grid_dependency_wait();
    tc::allow_dependents();
    const float share = 1.0f / (float)a.D;
    F2 s0[M][PAIRS], s1[M][PAIRS];  // of the thread's channels over its rows: dz, dz hat
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) s0[m][i] = s1[m][i] = f2(0.0f);
    Word ww[M], wb[M], next_x[M], next_d[M];
    float2 next_st = make_float2(0.0f, 0.0f);
    auto fetch = [&](int64_t n) {
        fetch_row(a, at, a.x, n, next_x);
        fetch_row(a, at, a.dy, n, next_d);
        if (at.in && n < a.N) next_st = reinterpret_cast<const float2 *>(a.stats)[n * a.G + at.g];
    };
    constexpr bool AHEAD = M <= 2;  // (as above: four spilled 520 bytes)
    if (AHEAD) fetch(at.n);
    fetch_row(a, at, a.w, 0, ww);
    fetch_row(a, at, a.b, 0, wb);
    with_norm_act(a.act, [&](auto kind) {
        for (int64_t n = at.n; n - at.row < a.N; n += at.step) {
            const bool there = at.in && n < a.N;
            if (!AHEAD) fetch(n);
            const float2 st = next_st;
            Word wx[M], wd[M];
#pragma unroll
            for (int m = 0; m < M; ++m) wx[m] = next_x[m], wd[m] = next_d[m];
            if (AHEAD) fetch(n + at.step);
            F2 hat[M][PAIRS], e[M][PAIRS];  // e: w dz
            float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (!there || !at.has(m)) continue;
                F2 w[PAIRS], b[PAIRS];
                params_of<T, V>(a.w, ww[m], 1.0f, w);
                params_of<T, V>(a.b, wb[m], 0.0f, b);
                to_pairs<T, V>(wx[m], hat[m]);
                to_pairs<T, V>(wd[m], e[m]);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    hat[m][i] = mul2(add2(hat[m][i], f2(-st.x)), f2(st.y));
                    const F2 dz = mul2(e[m][i], slope_of<T, decltype(kind)::value>(fma2(hat[m][i], w[i], b[i])));
                    s0[m][i] = add2(s0[m][i], dz);
                    s1[m][i] = fma2(dz, hat[m][i], s1[m][i]);
                    e[m][i] = mul2(dz, w[i]);
                    t0 += pair_sum<V>(e[m][i]);
                    t1 += pair_sum<V>(mul2(e[m][i], hat[m][i]));
                }
            }
            if (!a.dx) continue;  // (of every thread alike)
            const F2 m1 = f2(-at.sum(t0) * share), m2 = f2(-at.sum(t1) * share);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (!there || !at.has(m)) continue;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) e[m][i] = mul2(fma2(hat[m][i], m2, add2(e[m][i], m1)), f2(st.y));
                *reinterpret_cast<Word *>(static_cast<T *>(a.dx) + n * a.C + at.channel(a, m)) = from_pairs<T, V>(e[m]);
            }
        }
    });
    if (!a.dw && !a.db) return;
    // over the block's rows, one after the other
#pragma unroll
    for (int m = 0; m < M; ++m) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) red[2 * i][threadIdx.x] = s0[m][i], red[2 * i + 1][threadIdx.x] = s1[m][i];
        __syncthreads();
        if (at.row > 0 || !at.in || !at.has(m)) continue;
        for (int r = 1; r < a.rows; ++r)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                s0[m][i] = add2(s0[m][i], red[2 * i][threadIdx.x + r * a.cols]);
                s1[m][i] = add2(s1[m][i], red[2 * i + 1][threadIdx.x + r * a.cols]);
            }
        store_channels<V>(a, blockIdx.x / a.slabs, at.channel(a, m), s0[m], s1[m]);
    }
}

template <typename K, typename... A>
cudaError_t launch_with(K kernel, int64_t blocks, cudaStream_t st, int smem, int cluster, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = smem;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename K>
cudaError_t launch(K kernel, int64_t blocks, cudaStream_t st, const GroupArgs &a, int smem = 0, int cluster = 1) {
    return launch_with(kernel, blocks, st, smem, cluster, a);
}

// A block a group where a warp would take more than 8 loads of each sum.
inline bool by_block(const GroupArgs &a) { return (int64_t)a.D * a.chunks > 256; }
inline int64_t group_blocks(const GroupArgs &a) { return by_block(a) ? a.N * a.G : (a.N * a.G + 7) / 8; }

template <typename T, typename Fn>
cudaError_t with_vector(const GroupArgs &a, Fn f) {
    switch (vector_of(a.C, sizeof(T))) {
        case 1: return f(IntC<1>());
        case 2: return f(IntC<2>());
        default: return f(IntC<16 / (int)sizeof(T)>());
    }
}

// Calls f with the vector of a group's elements and a thread's number of them.
template <typename T, typename Fn>
cudaError_t with_row_vectors(const GroupArgs &a, Fn f) {
    const int v = vector_of(a.D, sizeof(T)), m = (a.D / v + a.lanes - 1) / a.lanes;
    auto go = [&](auto vec) { return m == 1 ? f(vec, IntC<1>()) : m == 2 ? f(vec, IntC<2>()) : f(vec, IntC<4>()); };
    return v == 1 ? go(IntC<1>()) : v == 2 ? go(IntC<2>()) : go(IntC<16 / (int)sizeof(T)>());
}

}  // namespace

template <typename T>
cudaError_t launch_forward(const GroupArgs &a, cudaStream_t st) {
    if (a.lanes)
        return with_row_vectors<T>(a, [&](auto v, auto m) {
            return launch(gn_rows<T, decltype(v)::value, decltype(m)::value>, a.slabs * a.chunks, st, a);
        });
    const int64_t blocks = a.N * a.slabs * a.chunks;
    return with_vector<T>(a, [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (a.resident) {
            const cudaError_t e = allow_smem<gn_resident<T, V>>(MAX_SMEM);
            return e == cudaSuccess ? launch(gn_resident<T, V>, blocks, st, a, a.smem, a.chunks) : e;
        }
        cudaError_t e = launch(gn_moments<T, V>, blocks, st, a);
        // (eight lanes for 64 items: 200704 images of 4 x 64 in eight groups take 1880 us, 2350 us with 32)
        if (e == cudaSuccess)
            e = by_block(a)                 ? launch(gn_stats<THREADS>, a.N * a.G, st, a)
                : a.D * a.chunks > 64       ? launch(gn_stats<32>, (a.N * a.G + 7) / 8, st, a)
                                            : launch(gn_stats<8>, (a.N * a.G + 31) / 32, st, a);
        return e == cudaSuccess ? launch(gn_apply<T, V>, blocks, st, a) : e;
    });
}

template <typename T>
cudaError_t launch_backward(const GroupArgs &a, cudaStream_t st) {
    const int params = a.dw || a.db ? (a.C + 31) / 32 : 0;
    auto sum = [&](cudaError_t e) { return e == cudaSuccess && params ? launch(gn_back_params<T>, params, st, a) : e; };
    if (a.lanes) {
        cudaError_t e = with_row_vectors<T>(a, [&](auto v, auto m) {
            return launch(gn_back_rows<T, decltype(v)::value, decltype(m)::value>, a.slabs * a.chunks, st, a);
        });
        return sum(e);
    }
    const int64_t blocks = a.N * a.slabs * a.chunks;
    return with_vector<T>(a, [&](auto v) {
        constexpr int V = decltype(v)::value;
        cudaError_t e = a.resident ? allow_smem<gn_back_resident<T, V>>(MAX_SMEM) : cudaSuccess;
        if (e == cudaSuccess)
            e = a.resident ? launch(gn_back_resident<T, V>, blocks, st, a, a.smem, a.chunks) : launch(gn_back_sums<T, V>, blocks, st, a);
        if (e == cudaSuccess && params && a.folds) e = launch(gn_back_fold, (int64_t)params * a.folds, st, a);
        if (a.dx && !a.resident) {
            if (e == cudaSuccess)
                e = by_block(a) ? launch(gn_back_means<T, THREADS>, group_blocks(a), st, a) : launch(gn_back_means<T, 32>, group_blocks(a), st, a);
            // dw and db beside dx, if the grid holds both
            const int beside = blocks + params <= 0x7fffffff ? params : 0;
            if (e == cudaSuccess) e = launch_with(gn_back_apply<T, V>, blocks + beside, st, 0, 1, a, beside);
            return beside ? e : sum(e);
        }
        return sum(e);
    });
}

}  // namespace gnorm
}  // namespace im2win
