// What the experts' products need before and after them: the plan (a stable counting sort of
// the pairs by expert), the rows gathered by expert, and the sums of a row's weighted outputs.
//
// Nothing here depends on the order of blocks: a pair's place is the number of its expert's
// pairs before it, and sums run over a row's choices in their order. The plan of 25088 pairs takes 7 us, of 1554
// 5 us (one block: a chain of barriers and dependent loads); gathering and summing run at the memory's rate (16384
// pairs of 2048 channels: 19 us, 38 us with the products dy . ys, 27 us).
#include <algorithm>
#include <type_traits>

#include "expert_ffn.cuh"
#include "tc_ptx.cuh"

namespace im2win {
namespace ffn {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr unsigned ALL = 0xffffffffu;

__global__ void __launch_bounds__(THREADS) expert_count(const int32_t *experts, int32_t *hist, int64_t pairs, int per, int E) {
    __shared__ int32_t sum[MAX_EXPERTS];
    tc::grid_dependency_wait();
    tc::allow_dependents();
    for (int e = threadIdx.x; e < E; e += THREADS) sum[e] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * per, end = min(pairs, begin + per);
    for (int64_t q = begin + threadIdx.x; q < end; q += THREADS) {
        const int32_t e = experts[q];
        if ((uint32_t)e < (uint32_t)E) atomicAdd(&sum[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += THREADS) hist[(int64_t)blockIdx.x * E + e] = sum[e];
}

constexpr int PLACE_THREADS = 1024, PLACE_WARPS = PLACE_THREADS / 32;

// Each warp takes a run of the block's pairs: it counts them by expert, and when the counts of the blocks and
// warps before it are known, gives them their rows in their order.
__global__ void __launch_bounds__(PLACE_THREADS) expert_place(const int32_t *experts, const int32_t *hist, int64_t pairs,
                                                              int per, int E, PairPlan plan, uint32_t *status) {
    extern __shared__ int32_t next[];  // [PLACE_WARPS][E]: counts, then the warp's next rows
    __shared__ int32_t total[MAX_EXPERTS], first[MAX_EXPERTS];
    // (not before the wait: the products that follow take tensor memory as soon as they start)
    tc::grid_dependency_wait();
    tc::allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x;
    const int run = (per + PLACE_WARPS - 1) / PLACE_WARPS;
    const int64_t block_end = min(pairs, (int64_t)(b + 1) * per), begin = min(block_end, (int64_t)b * per + (int64_t)warp * run),
                  end = min(block_end, begin + run);
    int32_t *mine = next + warp * E;
    if (b == 0 && threadIdx.x == 0) status[0] = 0;
    for (int e = lane; e < E; e += 32) mine[e] = 0;
    __syncwarp();
    for (int64_t q = begin + lane; q < end; q += 32) {
        const int32_t e = experts[q];
        if ((uint32_t)e < (uint32_t)E) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += PLACE_THREADS) {
        int32_t before = 0, sum = 0;  // the expert's pairs in the blocks before, and in all
        if (hist) {
#pragma unroll 8
            for (int i = 0; i < (int)gridDim.x; ++i) {
                const int32_t v = hist[(int64_t)i * E + e];
                before += i < b ? v : 0;
                sum += v;
            }
        }
#pragma unroll 8
        for (int w = 0; w < PLACE_WARPS; ++w) {
            const int32_t v = next[w * E + e];
            next[w * E + e] = before;
            before += v;
        }
        total[e] = hist ? sum : before;
    }
    __syncthreads();
    if (warp == 0) {
        int rows = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, padded = e < E ? (total[e] + GROUP_ROWS - 1) / GROUP_ROWS * GROUP_ROWS : 0;
            int sum = padded;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(ALL, sum, o);
                if (lane >= o) sum += v;
            }
            if (e < E) first[e] = rows + sum - padded;
            rows += __shfl_sync(ALL, sum, 31);
        }
        if (b == 0 && lane == 0) plan.begin[E] = rows;
    }
    __syncthreads();
    if (b == 0) {
        for (int e = warp; e < E; e += PLACE_WARPS) {
            if (lane == 0) plan.begin[e] = first[e], plan.count[e] = total[e];
            const int padded = (total[e] + GROUP_ROWS - 1) / GROUP_ROWS * GROUP_ROWS;
            for (int i = total[e] + lane; i < padded; i += 32) plan.pair[first[e] + i] = -1;
        }
    }
    for (int64_t q0 = begin; q0 < end; q0 += 32) {
        const int64_t q = q0 + lane;
        int32_t e = q < end ? experts[q] : -1;
        if ((uint32_t)e >= (uint32_t)E) e = -1;
        const unsigned same = __match_any_sync(ALL, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (e >= 0) {
            const int row = first[e] + mine[e] + rank;
            plan.slot[q] = row;
            plan.pair[row] = (int32_t)q;
        } else if (q < end) {
            plan.slot[q] = -1;
        }
        __syncwarp();
        if (rank == 0 && e >= 0) mine[e] += __popc(same);
        __syncwarp();
    }
}

// Eight elements from p on, `n` of them there; V: whole, aligned vectors.
template <typename T, bool V>
__device__ __forceinline__ void load8(const T *p, int n, float (&v)[8]) {
    if constexpr (V) {
#pragma unroll
        for (int i = 0; i < 8 * (int)sizeof(T) / 16; ++i) {
            const Vec16<T> w = reinterpret_cast<const Vec16<T> *>(p)[i];
#pragma unroll
            for (int j = 0; j < Vec16<T>::N; ++j) v[i * Vec16<T>::N + j] = to_f32(w.v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
    }
}
template <typename T, bool V>
__device__ __forceinline__ void store8(T *p, int n, const float (&v)[8]) {
    if constexpr (V) {
#pragma unroll
        for (int i = 0; i < 8 * (int)sizeof(T) / 16; ++i) {
            Vec16<T> w;
#pragma unroll
            for (int j = 0; j < Vec16<T>::N; ++j) w.v[j] = from_f32<T>(v[i * Vec16<T>::N + j]);
            reinterpret_cast<Vec16<T> *>(p)[i] = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
}
// Eight elements of a grouped row: an operand of the products, with whole vectors.
template <typename T>
__device__ __forceinline__ void store_operand(void *grouped, const Rows &r, int64_t row, int c, const float (&v)[8]) {
    const int64_t at = row * r.Cp + c;
    if constexpr (sizeof(T) == 2) {
        store8<T, true>(static_cast<T *>(grouped) + at, 8, v);
    } else {
        uint16_t *planes = static_cast<uint16_t *>(grouped) + at;
        alignas(16) uint16_t h[3][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split_f32(v[i], h[0][i], h[1][i], h[2][i]);
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4 *>(planes + q * r.rows * r.Cp) = *reinterpret_cast<const uint4 *>(h[q]);
    }
}
// The grouped row's pair: -1 in the padding, -2 past the last row.
__device__ __forceinline__ int64_t pair_of(const Rows &r, int64_t row) {
    if (row >= r.rows || row >= r.plan.begin[r.E]) return -2;
    const int64_t q = r.plan.pair[row];
    return q < 0 || q >= r.T * r.k ? -1 : q;
}

// A warp for 256 * GATHER columns of a row: looking up where the row comes from takes longer than copying 256, but
// registers for 1024 of which most are not there cost more (2048 columns: 24 us and 31 us; 256: 15 us and 12 us).
template <typename T, bool V, int GATHER>
__global__ void __launch_bounds__(THREADS) expert_gather(const __grid_constant__ Rows r, const T *x, const T *weights,
                                                         void *grouped, float *scale, int parts) {
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t id = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5), row = id / parts;
    const int c0 = ((int)(id - row * parts) * GATHER * 32 + (threadIdx.x & 31)) * 8;
    const int64_t q = pair_of(r, row);
    if (q < -1) return;
    if (scale && c0 == 0) scale[row] = q >= 0 ? to_f32(weights[q]) : 0.0f;
    const T *from = x + (q >= 0 ? q / r.k * r.C : 0);
    float v[GATHER][8] = {};
#pragma unroll
    for (int i = 0; i < GATHER; ++i) {
        const int c = c0 + i * 256;
        if (q >= 0 && c < r.Cp) load8<T, V>(from + c, r.C - c, v[i]);
    }
#pragma unroll
    for (int i = 0; i < GATHER; ++i)
        if (c0 + i * 256 < r.Cp) store_operand<T>(grouped, r, row, c0 + i * 256, v[i]);
}

// A warp a row.
template <typename T, bool V>
__global__ void __launch_bounds__(THREADS) expert_gather_back(const __grid_constant__ Rows r, const T *dy, const T *weights,
                                                              const float *ys, void *grouped, float *scale, T *dweights,
                                                              uint32_t *status) {
    tc::grid_dependency_wait();
    tc::allow_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) status[0] = 0;
    const int64_t id = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (dweights && id < r.T * r.k && r.plan.slot[id] < 0) dweights[id] = from_f32<T>(0.0f);
    const int64_t row = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5), q = pair_of(r, row);
    if (q < -1) return;
    if ((threadIdx.x & 31) == 0) scale[row] = q >= 0 ? to_f32(weights[q]) : 0.0f;
    const T *from = dy + (q >= 0 ? q / r.k * r.C : 0);
    float dot = 0.0f;
    for (int c = (threadIdx.x & 31) * 8; c < r.Cp; c += 256) {
        float d[8] = {};
        if (q >= 0) {
            load8<T, V>(from + c, r.C - c, d);
            if (dweights) {
                float o[8];
                load8<float, true>(ys + row * r.Cp + c, 8, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = c + i < r.C ? fmaf(d[i], o[i], dot) : dot;
            }
        }
        store_operand<T>(grouped, r, row, c, d);
    }
    if (!dweights || q < 0) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(ALL, dot, o);
    if ((threadIdx.x & 31) == 0) dweights[q] = from_f32<T>(dot);
}

// A warp for 256 columns of an output row.
template <typename T, bool V>
__global__ void __launch_bounds__(THREADS) expert_combine(const __grid_constant__ Rows r, const float *ys, const T *weights,
                                                          T *out, int parts) {
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t id = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5), t = id / parts;
    const int c = ((int)(id - t * parts) * 32 + (threadIdx.x & 31)) * 8;
    if (t >= r.T || c >= r.C) return;
    float sum[8] = {};
#pragma unroll 2
    for (int j = 0; j < r.k; ++j) {
        const int64_t slot = r.plan.slot[t * r.k + j];
        if (slot < 0 || slot >= r.rows) continue;
        float v[8];
        load8<float, true>(ys + slot * r.Cp + c, 8, v);
        const float w = weights ? to_f32(weights[t * r.k + j]) : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, v[i], sum[i]);
    }
    store8<T, V>(out + t * r.C + c, r.C - c, sum);
}

template <typename K, typename... A>
cudaError_t launch_sized(K kernel, int64_t blocks, int threads, int smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename K, typename... A>
cudaError_t launch(K kernel, int64_t blocks, cudaStream_t st, A... args) {
    return launch_sized(kernel, blocks, THREADS, 0, st, args...);
}

// Calls f with null pointers of the type, and whether rows of C are whole vectors.
template <typename Fn>
cudaError_t with_rows(int dtype, int C, Fn f) {
    cudaError_t e = cudaErrorInvalidValue;
    with_dtype(dtype, [&](auto *t) {
        e = C % 8 == 0 ? f(t, std::true_type()) : f(t, std::false_type());
    });
    return e;
}

}  // namespace

cudaError_t launch_plan(const Rows &r, const int32_t *experts, int32_t *hist, uint32_t *status, cudaStream_t st) {
    const int64_t pairs = r.T * r.k;
    const int per = (int)pairs_per_block(pairs);
    const int64_t blocks = (pairs + per - 1) / per;
    cudaError_t e = cudaSuccess;
    if (blocks > 1) e = launch(expert_count, blocks, st, experts, hist, pairs, per, r.E);
    if (e != cudaSuccess) return e;
    const int smem = PLACE_WARPS * r.E * 4;
    e = allow_smem<expert_place>(PLACE_WARPS * MAX_EXPERTS * 4);
    if (e != cudaSuccess) return e;
    return launch_sized(expert_place, blocks, PLACE_THREADS, smem, st, experts,
                        static_cast<const int32_t *>(blocks > 1 ? hist : nullptr), pairs, per, r.E, r.plan, status);
}

cudaError_t launch_gather(const Rows &r, const void *x, const void *weights, void *grouped, float *scale, int dtype,
                          cudaStream_t st) {
    const int columns = r.Cp <= 512 ? 256 : 1024, parts = (int)((r.Cp + columns - 1) / columns);
    return with_rows(dtype, r.C, [&](auto *t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr bool V = decltype(v)::value;
        return launch(columns == 256 ? expert_gather<T, V, 1> : expert_gather<T, V, 4>, (r.rows * parts + WARPS - 1) / WARPS, st, r,
                      static_cast<const T *>(x), static_cast<const T *>(weights), grouped, scale, parts);
    });
}

cudaError_t launch_gather_back(const Rows &r, const void *dy, const void *weights, const float *ys, void *grouped,
                               float *scale, void *dweights, uint32_t *status, int dtype, cudaStream_t st) {
    return with_rows(dtype, r.C, [&](auto *t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        return launch(expert_gather_back<T, decltype(v)::value>, (r.rows + WARPS - 1) / WARPS, st, r, static_cast<const T *>(dy),
                      static_cast<const T *>(weights), ys, grouped, scale, static_cast<T *>(dweights), status);
    });
}

cudaError_t launch_combine(const Rows &r, const float *ys, const void *weights, void *out, int dtype, cudaStream_t st) {
    const int parts = (r.C + 255) / 256;
    return with_rows(dtype, r.C, [&](auto *t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        return launch(expert_combine<T, decltype(v)::value>, (r.T * parts + WARPS - 1) / WARPS, st, r,
                      ys, static_cast<const T *>(weights), static_cast<T *>(out), parts);
    });
}

}  // namespace ffn
}  // namespace im2win
