// Global norm of a list of gradients and their clipping, in two launches for
// each table of tensors: sums of squares, one partial for each block, and the
// scaling, whose every block joins the partials in the same order while its first
// gradients are on their way.
//
// Bound by memory: two readings and one writing (lists that L2 holds: one of
// each). 1.5 G values of 48 bf16 and fp32 tensors, 3 GB: 1384 us, 6.5 TB/s through
// the three passes; 3.2 M fp32 values of 53: 13 us. 16-byte vectors, 8192 elements of
// one tensor a block at a time, whose loads are all under way before the first is
// used; four blocks an SM, with registers for that (eight: 1425 us).
//
// Squares and their sum in a thread are fp32 (32 values), sums over chunks, threads
// and blocks fp64, the last two by one warp of a block: the fp64 units are few (by every warp,
// with the factor in fp64 too, the 3.2 M values took 25 us).
#include <algorithm>
#include <cmath>

#include "elem.cuh"
#include "tc_ptx.cuh"

using namespace im2win;

namespace {

constexpr int THREADS = 256;
constexpr int CHUNK = 8192;  // elements a block takes at a time, all of one tensor
constexpr int PARTS = 608;   // blocks and partial sums of a table at most (4 on each of 152 SMs)

struct Entry {
    const void *in;
    void *out;
    int64_t size;
    uint32_t first;  // the tensor's first chunk
    int dtype;
};

// The tensors of one launch, passed in its parameters; `first` of entry `count`
// would be `chunks`.
template <int CAP>
struct Table {
    int count;
    uint32_t chunks;
    Entry e[CAP];
};
constexpr int SMALL = 64, LARGE = 960;  // 2 KB, 30 KB of parameters

template <int CAP>
__device__ __forceinline__ int entry_of(const Table<CAP> &t, uint32_t chunk) {
    int lo = 0, hi = t.count;  // the last entry whose first chunk is <= chunk
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.e[mid].first <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A thread's sum of squares `a`, or, where they passed fp32's range (its subnormal numbers,
// which the sums below 2^-100 may hold, or its largest), the same of the values times a power
// of two: again(scale).
template <typename Fn>
__device__ __forceinline__ double in_range(float a, Fn again) {
    if (a >= 0x1p-100f && a <= 3.402823466e38f) return a;
    const bool large = !(a < 1.0f);  // (infinite, or NaN)
    return (double)again(large ? 0x1p-100f : 0x1p100f) * (large ? 0x1p200 : 0x1p-200);
}

template <typename T>
__device__ __forceinline__ double squares(const T *p, int n) {
    using V = Vec16<T>;
    auto add = [](float &a, const V &v, float scale) {
#pragma unroll
        for (int j = 0; j < V::N; ++j) {
            const float x = to_f32(v.v[j]) * scale;
            a = fmaf(x, x, a);
        }
    };
    const bool vectors = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    const V *from = reinterpret_cast<const V *>(p);
    if (vectors && n == CHUNK) {  // (without conditions: with them this loop has two thirds of the rate)
        V v[CHUNK / (THREADS * V::N)];
#pragma unroll
        for (int i = 0; i < CHUNK / (THREADS * V::N); ++i) v[i] = from[i * THREADS + threadIdx.x];
        auto sum = [&](float scale) {
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < CHUNK / (THREADS * V::N); ++i) add(a, v[i], scale);
            return a;
        };
        return in_range(sum(1.0f), sum);
    }
    const int done = vectors ? n / V::N * V::N : 0;
    auto sum = [&](float scale) {
        float a = 0.0f;
#pragma unroll 4
        for (int i = threadIdx.x; i < done / V::N; i += THREADS) add(a, from[i], scale);
        for (int i = done + threadIdx.x; i < n; i += THREADS) {
            const float x = to_f32(p[i]) * scale;
            a = fmaf(x, x, a);
        }
        return a;
    };
    return in_range(sum(1.0f), sum);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int CAP>
__global__ void __launch_bounds__(THREADS, 4) sum_squares(const __grid_constant__ Table<CAP> t, double *part) {
    tc::allow_dependents();
    __shared__ double sums[THREADS];
    double a = 0.0;
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry &e = t.e[entry_of(t, c)];
        const int64_t at = (int64_t)(c - e.first) * CHUNK;
        const int n = (int)min((int64_t)CHUNK, e.size - at);
        if (e.dtype == IM2WIN_F32) a += squares(static_cast<const float *>(e.in) + at, n);
        else if (e.dtype == IM2WIN_F16) a += squares(static_cast<const f16_t *>(e.in) + at, n);
        else a += squares(static_cast<const bf16_t *>(e.in) + at, n);
    }
    sums[threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.x >= 32) return;
#pragma unroll
    for (int i = 1; i < THREADS / 32; ++i) a += sums[i * 32 + threadIdx.x];
    a = warp_sum(a);
    if (threadIdx.x == 0) part[blockIdx.x] = a;
}

// The norm and the factor of all gradients, from the partial sums of the launches before.
struct Factor {
    const double *part;
    int64_t parts;
    double max_norm, eps;
    float *norm;
    __device__ float get() const {
        __shared__ float f;
        tc::grid_dependency_wait();
        if (threadIdx.x < 32) {
            double a = 0.0;
#pragma unroll 8
            for (int64_t i = threadIdx.x; i < parts; i += 32) a += part[i];
            a = warp_sum(a);
            if (threadIdx.x == 0) {
                float total = sqrtf((float)a);
                if (!(a > 1e-30 && a < 1e38)) total = (float)sqrt(a);
                if (norm && blockIdx.x == 0) *norm = total;
                const float limit = (float)max_norm / (total + (float)eps);
                f = limit >= 1.0f ? 1.0f : limit;  // NaN stays NaN
            }
        }
        __syncthreads();
        return f;
    }
};

// FIRST: of a block's chunks, whose factor is asked for once its loads are under way.
template <bool FIRST, typename T>
__device__ __forceinline__ void scale(const T *in, T *out, int n, float &f, const Factor &factor) {
    using V = Vec16<T>;
    auto times = [&](V &v) {
#pragma unroll
        for (int j = 0; j < V::N; ++j) v.v[j] = from_f32<T>(to_f32(v.v[j]) * f);
    };
    const bool vectors = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const V *from = reinterpret_cast<const V *>(in);
    V *to = reinterpret_cast<V *>(out);
    if (vectors && n == CHUNK) {
        V v[CHUNK / (THREADS * V::N)];
#pragma unroll
        for (int i = 0; i < CHUNK / (THREADS * V::N); ++i) v[i] = from[i * THREADS + threadIdx.x];
        if (FIRST) f = factor.get();
        if (f == 1.0f && in == out) return;
#pragma unroll
        for (int i = 0; i < CHUNK / (THREADS * V::N); ++i) {
            times(v[i]);
            to[i * THREADS + threadIdx.x] = v[i];
        }
        return;
    }
    if (FIRST) f = factor.get();
    if (f == 1.0f && in == out) return;
    const int done = vectors ? n / V::N * V::N : 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < done / V::N; i += THREADS) {
        V v = from[i];
        times(v);
        to[i] = v;
    }
    for (int i = done + threadIdx.x; i < n; i += THREADS) out[i] = from_f32<T>(to_f32(in[i]) * f);
}

template <bool FIRST, int CAP>
__device__ __forceinline__ void scale_chunk(const Table<CAP> &t, uint32_t c, float &f, const Factor &factor) {
    const Entry &e = t.e[entry_of(t, c)];
    if (!FIRST && f == 1.0f && e.out == e.in) return;
    const int64_t at = (int64_t)(c - e.first) * CHUNK;
    const int n = (int)min((int64_t)CHUNK, e.size - at);
    if (e.dtype == IM2WIN_F32)
        scale<FIRST>(static_cast<const float *>(e.in) + at, static_cast<float *>(e.out) + at, n, f, factor);
    else if (e.dtype == IM2WIN_F16)
        scale<FIRST>(static_cast<const f16_t *>(e.in) + at, static_cast<f16_t *>(e.out) + at, n, f, factor);
    else
        scale<FIRST>(static_cast<const bf16_t *>(e.in) + at, static_cast<bf16_t *>(e.out) + at, n, f, factor);
}

template <int CAP>
__global__ void __launch_bounds__(THREADS, 4) clip(const __grid_constant__ Table<CAP> t, const Factor factor) {
    float f = 1.0f;
    uint32_t c = blockIdx.x;
    if (c < t.chunks) scale_chunk<true>(t, c, f, factor);
    else factor.get();
    while ((c += gridDim.x) < t.chunks) scale_chunk<false>(t, c, f, factor);
}
__global__ void __launch_bounds__(THREADS) norm_alone(const Factor factor) {
    factor.get();
}

int64_t tables(int64_t count) { return std::max<int64_t>(1, (count + LARGE - 1) / LARGE); }

// Entries [first, first + t.count) of the lists.
template <int CAP>
bool fill(Table<CAP> &t, const void *const *grads, void *const *outs, const int64_t *sizes, const int *dtypes,
          int64_t first, int64_t count) {
    t.count = (int)std::min<int64_t>(CAP, count - first);
    uint64_t chunks = 0;
    for (int i = 0; i < t.count; ++i) {
        Entry &e = t.e[i];
        e.in = grads[first + i];
        e.out = outs ? outs[first + i] : nullptr;
        e.size = sizes[first + i];
        e.dtype = dtypes[first + i];
        e.first = (uint32_t)chunks;
        chunks += (uint64_t)(e.size + CHUNK - 1) / CHUNK;
        if (chunks > 0x7fffffff) return false;
    }
    t.chunks = (uint32_t)chunks;
    return true;
}

unsigned blocks_of(uint32_t chunks) { return std::max(1u, std::min<unsigned>(chunks, PARTS)); }

template <int CAP>
im2win_status run(const void *const *grads, void *const *outs, const int64_t *sizes, const int *dtypes, int64_t count,
                  double max_norm, double eps, float *norm, double *part, cudaStream_t st) {
    static thread_local Table<CAP> t;
    const int64_t n_tables = tables(count);
    int64_t parts = 0;
    for (int64_t k = 0; k < n_tables; ++k) {
        if (!fill(t, grads, outs, sizes, dtypes, k * CAP, count)) return IM2WIN_ERR_UNSUPPORTED;
        const unsigned blocks = blocks_of(t.chunks);
        sum_squares<CAP><<<blocks, THREADS, 0, st>>>(t, part + parts);
        if (cudaGetLastError() != cudaSuccess) return IM2WIN_ERR_CUDA;
        parts += blocks;
    }
    // (the first of them begins while the last sums end; the others' inputs and outputs are other tensors)
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    for (int64_t k = 0; k < n_tables; ++k) {
        if (n_tables > 1) fill(t, grads, outs, sizes, dtypes, k * CAP, count);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(outs ? blocks_of(t.chunks) : 1);
        cfg.blockDim = dim3(THREADS);
        cfg.stream = st;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        const Factor factor = {part, parts, max_norm, eps, k == 0 ? norm : nullptr};
        const cudaError_t e = !outs ? cudaLaunchKernelEx(&cfg, norm_alone, factor)
                              : cudaLaunchKernelEx(&cfg, clip<CAP>, t, factor);
        if (e != cudaSuccess) return IM2WIN_ERR_CUDA;
        if (!outs) break;
    }
    return IM2WIN_OK;
}

}  // namespace

extern "C" {

im2win_status im2win_clip_grad_norm_size(const int64_t *sizes, int64_t count, size_t *bytes) {
    if (!bytes || count < 0 || (count > 0 && !sizes)) return IM2WIN_ERR_INVALID_ARG;
    if (count > (1 << 24)) return IM2WIN_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < count; ++i)
        if (sizes[i] < 0) return IM2WIN_ERR_INVALID_ARG;
    *bytes = (size_t)tables(count) * PARTS * sizeof(double);
    return IM2WIN_OK;
}

im2win_status im2win_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *sizes,
                                    const int *dtypes, int64_t count, double max_norm, double eps, float *norm,
                                    void *ws, size_t ws_bytes, void *stream) {
    size_t need = 0;
    const im2win_status s = im2win_clip_grad_norm_size(sizes, count, &need);
    if (s != IM2WIN_OK) return s;
    if (!norm || (count > 0 && (!grads || !dtypes)) || !(max_norm >= 0.0) || !(eps >= 0.0)) return IM2WIN_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i) {
        const int esz = elem_size(dtypes[i]);
        if (esz == 0) return IM2WIN_ERR_INVALID_ARG;
        if (sizes[i] == 0) continue;
        if (sizes[i] > (int64_t(1) << 40)) return IM2WIN_ERR_UNSUPPORTED;
        if (!grads[i] || (outs && !outs[i])) return IM2WIN_ERR_INVALID_ARG;
        if (!aligned_to(grads[i], esz) || (outs && !aligned_to(outs[i], esz))) return IM2WIN_ERR_MISALIGNED;
    }
    if (!ws || ws_bytes < need) return IM2WIN_ERR_WORKSPACE;
    if (!aligned_to(ws, 16) || !aligned_to(norm, 4)) return IM2WIN_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    double *part = static_cast<double *>(ws);
    return count <= SMALL ? run<SMALL>(grads, outs, sizes, dtypes, count, max_norm, eps, norm, part, st)
                          : run<LARGE>(grads, outs, sizes, dtypes, count, max_norm, eps, norm, part, st);
}

}  // extern "C"
