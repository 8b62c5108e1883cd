// The router: the k largest of a row of E logits and their softmax weights, and the gradient.
//
// A row belongs to L lanes with M neighbouring logits each, in registers; L and M are the
// smallest that hold E, so that few exchanges serve a row (64 experts: 8 lanes of 8, three
// exchanges a reduction; 8 experts: one thread a row). A choice is the largest key of
// the lanes' own largest, then the lowest lane that has it, which is the lowest index. The
// kernel reads the logits once. 50176 rows of 64 fp32 logits, four choices: 11 us forward, 9 us backward, bound by
// instructions (780 for a warp's four rows, 56% of the issue slots); 200704 rows of bf16, two choices: 22 us.
#include <algorithm>

#include "elem.cuh"
#include "tc_ptx.cuh"

using namespace im2win;

namespace {

constexpr int THREADS = 128;
constexpr int MAX_EXPERTS = 1024, MAX_K = 32;
constexpr unsigned ALL = 0xffffffffu;

struct RouteArgs {
    const void *logits, *dweights;
    void *weights, *dlogits;
    int32_t *experts;
    int64_t T;
    int E, k, over;
};

// Order of the logits as unsigned numbers: NaN above all, -infinity (an expert that may not
// be taken) zero, both zeros alike.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) return 0xffffffffu;
    if (v == -INFINITY) return 0u;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    if (key == 0xffffffffu) return __int_as_float(0x7fffffff);
    return key & 0x80000000u ? __uint_as_float(key & 0x7fffffffu) : key == 0u ? -INFINITY : __uint_as_float(~key);
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
    return v;
}
// The larger one; NaN if either is.
__device__ __forceinline__ float larger(float a, float b) { return a != a || a > b ? a : b; }
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = larger(v, __shfl_xor_sync(ALL, v, o));
    return v;
}

// The lane's M logits from index first on, -infinity past E; V: whole vectors of 16 bytes.
template <typename T, int M, bool V>
__device__ __forceinline__ void load_logits(const T *row, int first, int E, float (&l)[M]) {
    if constexpr (V) {
        constexpr int N = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < M / N; ++i) {
            if (first + i * N < E) {
                const Vec16<T> v = reinterpret_cast<const Vec16<T> *>(row + first)[i];
#pragma unroll
                for (int j = 0; j < N; ++j) l[i * N + j] = to_f32(v.v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) l[i * N + j] = -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i) l[i] = first + i < E ? to_f32(row[first + i]) : -INFINITY;
    }
}

template <typename T, int L, int M, bool V>
__global__ void __launch_bounds__(THREADS) route(const __grid_constant__ RouteArgs a) {
    __shared__ float chosen[THREADS / L][MAX_K + 1];  // exponentials of a row's choices
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t wanted = ((int64_t)blockIdx.x * THREADS + threadIdx.x) / L;
    const bool there = wanted < a.T;
    const int64_t t = there ? wanted : a.T - 1;  // (every lane takes part in the exchanges)
    const int lane = threadIdx.x % L, first = lane * M, begin = (int)(threadIdx.x & 31) / L * L;
    float *mine = chosen[threadIdx.x / L];
    float l[M];
    load_logits<T, M, V>(static_cast<const T *>(a.logits) + t * a.E, first, a.E, l);
    uint32_t key[M];
#pragma unroll
    for (int i = 0; i < M; ++i) key[i] = key_of(l[i]);
    float top = 0.0f, total = 0.0f;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < M; ++i)
            if (key[i] > best) best = key[i], at = i;
        uint32_t most = best;
        int e = first + at;
        bool owner = true;
        if constexpr (L > 1) {
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(ALL, most, o));
            const int from = __ffs(__ballot_sync(ALL, best == most) >> begin) - 1;
            e = __shfl_sync(ALL, e, from, L);
            owner = lane == from;
        }
        if (owner) {
#pragma unroll
            for (int i = 0; i < M; ++i)
                if (i == at) key[i] = 0u;
        }
        const float v = value_of(most);
        if (j == 0) {
            top = v;
            if (a.over == IM2WIN_ROUTE_ALL) {
#pragma unroll
                for (int i = 0; i < M; ++i) total += expf(l[i] - top);
                total = lanes_sum<L>(total);
            }
        }
        const float w = most == 0u ? 0.0f : expf(v - top);
        if (a.over == IM2WIN_ROUTE_TOP) total += w;
        if (lane == j % L) {
            mine[j] = w;
            if (there) a.experts[t * a.k + j] = most == 0u ? -1 : e;
        }
    }
    if (!there) return;
    // (a lane reads what it wrote; with no expert to take the total is zero or NaN)
    for (int j = lane; j < a.k; j += L) static_cast<T *>(a.weights)[t * a.k + j] = from_f32<T>(mine[j] == 0.0f ? 0.0f : mine[j] / total);
}

// dl of a row. TOP: w_j the softmax over the row's choices, dl_e = sum over j with e_j = e of
// w_j (dw_j - s), s = sum w_j dw_j. ALL: p the softmax over all, dl_e = p_e (sum of those dw_j - s),
// s = sum p_(e_j) dw_j.
template <typename T, int L, int M, bool V>
__global__ void __launch_bounds__(THREADS) route_backward(const __grid_constant__ RouteArgs a) {
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t wanted = ((int64_t)blockIdx.x * THREADS + threadIdx.x) / L;
    const bool there = wanted < a.T;
    const int64_t t = there ? wanted : a.T - 1;
    const int lane = threadIdx.x % L, first = lane * M;
    const T *row = static_cast<const T *>(a.logits) + t * a.E, *dweights = static_cast<const T *>(a.dweights) + t * a.k;
    const int32_t *experts = a.experts + t * a.k;
    const bool all = a.over == IM2WIN_ROUTE_ALL;
    float l[M];
    load_logits<T, M, V>(row, first, a.E, l);
    auto taken = [&](int j, int &e) {
        e = experts[j];
        return (unsigned)e < (unsigned)a.E;
    };
    float top = -INFINITY, total = 0.0f, s = 0.0f;
    if (all) {
#pragma unroll
        for (int i = 0; i < M; ++i) top = larger(top, l[i]);
    } else {
        for (int j = lane, e; j < a.k; j += L)
            if (taken(j, e)) top = larger(top, to_f32(row[e]));
    }
    top = lanes_max<L>(top);
    if (top == -INFINITY) top = 0.0f;  // (no expert to take: every exponential is zero)
    if (all) {
#pragma unroll
        for (int i = 0; i < M; ++i) total += l[i] = expf(l[i] - top);
    }
    for (int j = lane, e; j < a.k; j += L) {
        if (!taken(j, e)) continue;
        const float w = expf(to_f32(row[e]) - top);
        if (!all) total += w;
        s = fmaf(w, to_f32(dweights[j]), s);
    }
    total = lanes_sum<L>(total);
    if (total == 0.0f) total = 1.0f;
    s = lanes_sum<L>(s) / total;
    float d[M];
#pragma unroll
    for (int i = 0; i < M; ++i) d[i] = 0.0f;
    for (int j = 0, e; j < a.k; ++j) {
        if (!taken(j, e) || e < first || e >= first + M) continue;
        const float dw = to_f32(dweights[j]);
        const float add = all ? dw : expf(to_f32(row[e]) - top) / total * (dw - s);
#pragma unroll
        for (int i = 0; i < M; ++i)
            if (first + i == e) d[i] += add;
    }
    if (all) {
#pragma unroll
        for (int i = 0; i < M; ++i) d[i] = l[i] / total * (d[i] - s);
    }
    if (!there) return;
    T *out = static_cast<T *>(a.dlogits) + t * a.E + first;
    if constexpr (V) {
        constexpr int N = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < M / N; ++i) {
            if (first + i * N >= a.E) continue;
            Vec16<T> v;
#pragma unroll
            for (int j = 0; j < N; ++j) v.v[j] = from_f32<T>(d[i * N + j]);
            reinterpret_cast<Vec16<T> *>(out)[i] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < M; ++i)
            if (first + i < a.E) out[i] = from_f32<T>(d[i]);
    }
}

template <typename K>
cudaError_t launch(K kernel, int64_t blocks, cudaStream_t st, const RouteArgs &a) {
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

template <typename T, int L, int M>
cudaError_t launch_lanes(const RouteArgs &a, bool backward, cudaStream_t st) {
    const int64_t blocks = (a.T + THREADS / L - 1) / (THREADS / L);
    if (a.E % (16 / (int)sizeof(T)) == 0) return launch(backward ? route_backward<T, L, M, true> : route<T, L, M, true>, blocks, st, a);
    return launch(backward ? route_backward<T, L, M, false> : route<T, L, M, false>, blocks, st, a);
}

template <typename T>
cudaError_t launch_type(const RouteArgs &a, bool backward, cudaStream_t st) {
    if (a.E <= 8) return launch_lanes<T, 1, 8>(a, backward, st);
    if (a.E <= 16) return launch_lanes<T, 2, 8>(a, backward, st);
    if (a.E <= 32) return launch_lanes<T, 4, 8>(a, backward, st);
    if (a.E <= 64) return launch_lanes<T, 8, 8>(a, backward, st);
    if (a.E <= 128) return launch_lanes<T, 16, 8>(a, backward, st);
    if (a.E <= 256) return launch_lanes<T, 32, 8>(a, backward, st);
    return launch_lanes<T, 32, 32>(a, backward, st);
}

im2win_status check(int64_t T, int64_t E, int64_t k, int over, int dtype) {
    if (T < 0 || E < 1 || k < 1 || k > E || elem_size(dtype) == 0 || (over != IM2WIN_ROUTE_TOP && over != IM2WIN_ROUTE_ALL))
        return IM2WIN_ERR_INVALID_ARG;
    if (E > MAX_EXPERTS || k > MAX_K || T >= (int64_t(1) << 31)) return IM2WIN_ERR_UNSUPPORTED;
    return IM2WIN_OK;
}

im2win_status run(const RouteArgs &a, bool backward, int dtype, void *stream) {
    cudaError_t e = cudaErrorInvalidValue;
    with_dtype(dtype, [&](auto *t) {
        e = launch_type<std::remove_pointer_t<decltype(t)>>(a, backward, static_cast<cudaStream_t>(stream));
    });
    return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

}  // namespace

extern "C" {

im2win_status im2win_expert_route(const void *logits, void *weights, int32_t *experts, int64_t T, int64_t E, int64_t k,
                                  int over, int dtype, void *stream) {
    const im2win_status s = check(T, E, k, over, dtype);
    if (s != IM2WIN_OK || T == 0) return s;
    if (!logits || !weights || !experts) return IM2WIN_ERR_INVALID_ARG;
    if (!aligned_to(logits, 16) || !aligned_to(weights, elem_size(dtype)) || !aligned_to(experts, 4)) return IM2WIN_ERR_MISALIGNED;
    RouteArgs a = {};
    a.logits = logits, a.weights = weights, a.experts = experts;
    a.T = T, a.E = (int)E, a.k = (int)k, a.over = over;
    return run(a, false, dtype, stream);
}

im2win_status im2win_expert_route_backward(const void *dweights, const void *logits, const int32_t *experts,
                                           void *dlogits, int64_t T, int64_t E, int64_t k, int over, int dtype,
                                           void *stream) {
    const im2win_status s = check(T, E, k, over, dtype);
    if (s != IM2WIN_OK || T == 0) return s;
    if (!dweights || !logits || !experts || !dlogits) return IM2WIN_ERR_INVALID_ARG;
    if (!aligned_to(logits, 16) || !aligned_to(dlogits, 16) || !aligned_to(dweights, elem_size(dtype)) || !aligned_to(experts, 4))
        return IM2WIN_ERR_MISALIGNED;
    RouteArgs a = {};
    a.dweights = dweights, a.logits = logits, a.experts = const_cast<int32_t *>(experts), a.dlogits = dlogits;
    a.T = T, a.E = (int)E, a.k = (int)k, a.over = over;
    return run(a, true, dtype, stream);
}

}  // extern "C"
