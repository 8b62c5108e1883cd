// Global norm of a list of gradients and their clipping, in two launches for
// each table of tensors: sums of squares, one partial for each block, and the
// scaling, whose every block joins the partials in the same order.
//
// Bound by memory: two readings and one writing (lists that L2 holds: one of
// each). 1.5 G values of 48 bf16 and fp32 tensors, 3 GB: 1425 us, 6.6 TB/s through
// the three passes. 16-byte vectors, 8192 elements of one tensor a block at a time,
// whose loads are all under way before the first is used. Squares and their sum in
// a thread are fp32 (32 values), sums of threads and blocks fp64.
#include <algorithm>
#include <cmath>

#include "elem.cuh"

using namespace im2win;

namespace {

constexpr int THREADS = 256;
constexpr int CHUNK = 8192;  // elements a block takes at a time, all of one tensor
constexpr int PARTS = 1216;  // partial sums of a table (8 blocks on each of 152 SMs)

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

template <typename T>
__device__ __forceinline__ float squares(const T *p, int n) {
    float a = 0.0f;
    if (n == CHUNK && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        using V = Vec16<T>;
#pragma unroll
        for (int i = 0; i < CHUNK / (THREADS * V::N); ++i) {
            const V v = reinterpret_cast<const V *>(p)[i * THREADS + threadIdx.x];
#pragma unroll
            for (int j = 0; j < V::N; ++j) a = fmaf(to_f32(v.v[j]), to_f32(v.v[j]), a);
        }
    } else {
        for (int i = threadIdx.x; i < n; i += THREADS) a = fmaf(to_f32(p[i]), to_f32(p[i]), a);
    }
    return a;
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s[THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) t += s[i];
    __syncthreads();
    return t;
}

template <int CAP>
__global__ void __launch_bounds__(THREADS) sum_squares(const __grid_constant__ Table<CAP> t, double *part) {
    double a = 0.0;
    for (uint32_t c = blockIdx.x; c < t.chunks; c += PARTS) {
        const Entry &e = t.e[entry_of(t, c)];
        const int64_t at = (int64_t)(c - e.first) * CHUNK;
        const int n = (int)min((int64_t)CHUNK, e.size - at);
        if (e.dtype == IM2WIN_F32) a += squares(static_cast<const float *>(e.in) + at, n);
        else if (e.dtype == IM2WIN_F16) a += squares(static_cast<const f16_t *>(e.in) + at, n);
        else a += squares(static_cast<const bf16_t *>(e.in) + at, n);
    }
    a = block_sum(a);
    if (threadIdx.x == 0) part[blockIdx.x] = a;
}

template <typename T>
__device__ __forceinline__ void scale(const T *in, T *out, int n, float f) {
    if (n == CHUNK && ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
        using V = Vec16<T>;
        V v[CHUNK / (THREADS * V::N)];
#pragma unroll
        for (int i = 0; i < CHUNK / (THREADS * V::N); ++i)
            v[i] = reinterpret_cast<const V *>(in)[i * THREADS + threadIdx.x];
#pragma unroll
        for (int i = 0; i < CHUNK / (THREADS * V::N); ++i) {
#pragma unroll
            for (int j = 0; j < V::N; ++j) v[i].v[j] = from_f32<T>(to_f32(v[i].v[j]) * f);
            reinterpret_cast<V *>(out)[i * THREADS + threadIdx.x] = v[i];
        }
    } else {
        for (int i = threadIdx.x; i < n; i += THREADS) out[i] = from_f32<T>(to_f32(in[i]) * f);
    }
}

// `parts` partial sums of every table of the call.
template <int CAP>
__global__ void __launch_bounds__(THREADS)
    clip(const __grid_constant__ Table<CAP> t, const double *part, int64_t parts, double max_norm, double eps, float *norm) {
    double a = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += THREADS) a += part[i];
    const double total = sqrt(block_sum(a));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
    const double limit = max_norm / (total + eps);
    const float f = limit >= 1.0 ? 1.0f : (float)limit;  // NaN stays NaN
    for (uint32_t c = blockIdx.x; c < t.chunks; c += PARTS) {
        const Entry &e = t.e[entry_of(t, c)];
        if (e.out == nullptr || (f == 1.0f && e.out == e.in)) continue;
        const int64_t at = (int64_t)(c - e.first) * CHUNK;
        const int n = (int)min((int64_t)CHUNK, e.size - at);
        if (e.dtype == IM2WIN_F32) scale(static_cast<const float *>(e.in) + at, static_cast<float *>(e.out) + at, n, f);
        else if (e.dtype == IM2WIN_F16) scale(static_cast<const f16_t *>(e.in) + at, static_cast<f16_t *>(e.out) + at, n, f);
        else scale(static_cast<const bf16_t *>(e.in) + at, static_cast<bf16_t *>(e.out) + at, n, f);
    }
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

template <int CAP>
im2win_status run(const void *const *grads, void *const *outs, const int64_t *sizes, const int *dtypes, int64_t count,
                  double max_norm, double eps, float *norm, double *part, cudaStream_t st) {
    static thread_local Table<CAP> t;
    const int64_t n_tables = tables(count);
    for (int64_t k = 0; k < n_tables; ++k) {
        if (!fill(t, grads, outs, sizes, dtypes, k * CAP, count)) return IM2WIN_ERR_UNSUPPORTED;
        sum_squares<CAP><<<PARTS, THREADS, 0, st>>>(t, part + k * PARTS);
        if (cudaGetLastError() != cudaSuccess) return IM2WIN_ERR_CUDA;
    }
    for (int64_t k = 0; k < n_tables; ++k) {
        if (n_tables > 1) fill(t, grads, outs, sizes, dtypes, k * CAP, count);
        const unsigned grid = outs && t.chunks ? std::min<unsigned>(PARTS, t.chunks) : 1;
        clip<CAP><<<grid, THREADS, 0, st>>>(t, part, n_tables * PARTS, max_norm, eps, k == 0 ? norm : nullptr);
        if (cudaGetLastError() != cudaSuccess) return IM2WIN_ERR_CUDA;
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
