// The experts' feed-forward of few rows, bound by reading the chosen experts' weights once and by the
// number of its launches: two, without a plan, gathered rows or a sum of their own.
//
// The pairs of rows and experts are few enough for every block to sort them itself: those of an expert
// form groups of up to eight, the rows of a product on the gated feed-forward's scheme of few rows
// (16-bit types: 16 weight rows by mma.sync; fp32: 4 weight rows by FMA). The first launch takes
// (group, weight rows) after another over all SMs; an expert's further groups find its weights in L2. The
// second takes the weight rows of an output column for every group, adds the weighted products
// in the order of the groups and writes y; a cluster shares the groups where there are fewer
// columns than the SMs take, and joins its sums in the order of its CTAs.
//
// As there, h goes on as its rounding and the remainder of that (16-bit types), and what it makes stays
// in fp32 until y.
//
// One row by two of eight experts of 512 x 2048: 14 us (9 us of it in the two kernels); of 4096 x 10240 in bf16, 503
// MB: 114 us, 4.4 TB/s. fp32, 4 rows by two of eight of 2048 x 4096: 122 us.
#include <algorithm>
#include <type_traits>

#include "expert_ffn.cuh"
#include "ffn_few.cuh"

namespace im2win {
namespace ffn {
namespace {

constexpr int GROUP = 8;  // pairs of a group

struct ExpertFewParams {
    int T, k, E;
    int N, K;                   // weight rows of an expert; summed index
    const int32_t *experts;
    const void *weights;        // of the pairs (second launch)
    const void *b, *b_lo;       // x [T][ldb], or h and its remainder [T k][ldb]
    int64_t ldb;
    const void *w0, *w1;        // [E][N][K]; gate and up, or down alone
    int act;
    void *out, *out_lo;         // h and its remainder, or y
    int64_t ldo;
    int tiles, shares;          // of weight rows; CTAs of a cluster (second launch)
    uint32_t *status;           // cleared where not null
};

// The pairs in groups of an expert, in shared memory.
struct PairGroups {
    int n;                               // groups
    int expert[FEW_PAIRS], count[FEW_PAIRS];
    int pair[FEW_PAIRS][GROUP];
    int of[FEW_PAIRS], lead[FEW_PAIRS];  // each pair's expert; groups of the expert that it is the first of
};
__device__ __forceinline__ void sort_pairs(const ExpertFewParams &p, PairGroups &s) {
    const int pairs = p.T * p.k, i = threadIdx.x;
    int e = -1, first = i, rank = 0, count = 0;
    if (i < pairs) {
        e = p.experts[i];
        if ((uint32_t)e >= (uint32_t)p.E) e = -1;
        s.of[i] = e;
    }
    __syncthreads();
    if (i < pairs) {
        for (int j = pairs - 1; j >= 0; --j)
            if (s.of[j] == e) {
                ++count;
                if (j < i) ++rank;
                if (j < first) first = j;
            }
        s.lead[i] = e >= 0 && rank == 0 ? (count + GROUP - 1) / GROUP : 0;
    }
    __syncthreads();
    if (i < pairs) {
        int before = 0, all = 0;
        for (int j = 0; j < pairs; ++j) {
            before += j < first ? s.lead[j] : 0;
            all += s.lead[j];
        }
        if (i == 0) s.n = all;
        if (e >= 0) {
            const int g = before + rank / GROUP;
            s.pair[g][rank % GROUP] = i;
            if (rank % GROUP == 0) s.expert[g] = e, s.count[g] = min(GROUP, count - rank);
        }
    }
    __syncthreads();
}

// What a block works through: its groups and tiles, one after the other.
template <bool GATED>
struct Turn {
    int g, tile;
    __device__ Turn(const ExpertFewParams &p) {
        if (GATED) g = blockIdx.x / p.tiles, tile = blockIdx.x - g * p.tiles;
        else g = blockIdx.x % p.shares, tile = blockIdx.x / p.shares;
    }
    __device__ void next(const ExpertFewParams &p) {
        if (GATED) {
            tile += gridDim.x;
            if (tile >= p.tiles) g += tile / p.tiles, tile %= p.tiles;
        } else {
            g += p.shares;
        }
    }
};

// The second launch's sums of a block: ROWS columns of every row of y.
template <int COLS>
struct Outputs {
    float y[FEW_PAIRS][COLS];
    float part[GROUP][COLS];
};
// Adds a group's products, in part, weighted; every thread calls it, with part written before.
template <typename T, int COLS>
__device__ __forceinline__ void add_group(const ExpertFewParams &p, const PairGroups &s, Outputs<COLS> &o, int g) {
    __syncthreads();
    if (threadIdx.x < COLS) {
        for (int m = 0; m < s.count[g]; ++m) {  // (one after the other: a row may be there twice)
            const int q = s.pair[g][m];
            float &y = o.y[q / p.k][threadIdx.x];
            y = fmaf(to_f32(static_cast<const T *>(p.weights)[q]), o.part[m][threadIdx.x], y);
        }
    }
    __syncthreads();
}
// Joins the cluster's sums and writes y.
template <typename T, int COLS>
__device__ __forceinline__ void write_outputs(const ExpertFewParams &p, Outputs<COLS> &o, int tile) {
    const int rank = blockIdx.x % p.shares;
    if (p.shares > 1) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    for (int id = rank * THREADS + threadIdx.x; id < p.T * COLS; id += p.shares * THREADS) {
        const int t = id / COLS, c = id % COLS, n = tile * COLS + c;
        float sum = 0.0f;
        for (int r = 0; r < p.shares; ++r) {
            float v = o.y[t][c];
            if (p.shares > 1) {
                uint32_t at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(&o.y[t][c])), "r"(r));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
            }
            sum += v;
        }
        if (n < p.N) static_cast<T *>(p.out)[(int64_t)t * p.ldo + n] = from_f32<T>(sum);
    }
    // (no CTA may end while another reads its sums)
    if (p.shares > 1) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// 16-bit types. V: elements of the weights' vectors, VB: of b's.
template <bool BF16, int V, int VB, bool GATED>
__global__ void __launch_bounds__(THREADS, 2) expert_few_mma(const __grid_constant__ ExpertFewParams p) {
    using T = std::conditional_t<BF16, bf16_t, f16_t>;
    constexpr int NW = GATED ? 2 : 1, COLS = 16, TILE = COLS * GROUP, STEP = WARPS * 32;
    constexpr bool AHEAD = V == 8;
    using Stages = Ring<RING_VECS<1, GATED>>;
    extern __shared__ uint4 dyn[];
    __shared__ PairGroups s;
    __shared__ Outputs<GATED ? 1 : COLS> o;
    float *red = reinterpret_cast<float *>(dyn) + (AHEAD ? Stages::BYTES / 4 : 0);  // [WARPS][NW * TILE]
    Stages ring(dyn);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k_lane = warp * 32 + (lane % 4) * 8;
    // The second launch begins while the first runs, which has waited for all before it and writes h alone: the
    // pairs and the first weights need not wait for it.
    if (GATED) tc::grid_dependency_wait();
    tc::allow_dependents();
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;
    if (!GATED)
        for (int i = threadIdx.x; i < FEW_PAIRS * COLS; i += THREADS) (&o.y[0][0])[i] = 0.0f;
    sort_pairs(p, s);
    // weight row h (0, 1: eight rows apart) of the lane in matrix i, of a tile; the lane's row of b
    auto row = [&](const Turn<GATED> &t, int i, int h) {
        return static_cast<const uint16_t *>(i ? p.w1 : p.w0) +
               ((int64_t)s.expert[t.g] * p.N + min(t.tile * COLS + lane / 4 + h * 8, p.N - 1)) * p.K;
    };
    auto b_row = [&](const Turn<GATED> &t) {
        const int q = s.pair[t.g][min(lane / 4, s.count[t.g] - 1)];
        return (int64_t)(GATED ? q / p.k : q) * p.ldb;
    };
    const uint16_t *b = static_cast<const uint16_t *>(p.b), *b_lo = static_cast<const uint16_t *>(p.b_lo);
    auto copy_weights = [&](int stage, const Turn<GATED> &t, int k) {
        const bool in = k < p.K;
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) ring.copy(stage, i * 2 + h, row(t, i, h) + (in ? k : 0), in);
    };
    Turn<GATED> ahead(p);
    int ahead_k = 0;
    auto start = [&](int stage, bool weights) {
        if (!AHEAD) return;
        if (ahead.g < s.n) {
            const int k = ahead_k + k_lane;
            const bool in = k < p.K, there = in && lane / 4 < s.count[ahead.g];
            const int64_t at = in ? k : 0;
            if (weights) copy_weights(stage, ahead, k);
            const int64_t from = b_row(ahead) + at;
            ring.copy(stage, 2 * NW, b + from, there);
            if (!GATED) ring.copy(stage, 2 * NW + 1, b_lo + from, there);
            ahead_k += STEP;
            if (ahead_k >= p.K) ahead_k = 0, ahead.next(p);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (AHEAD && !GATED) {
        Turn<GATED> first(p);
        int k = 0;
#pragma unroll
        for (int i = 0; i < Stages::DEPTH - 1; ++i) {
            if (first.g < s.n) copy_weights(i, first, k + k_lane);
            k += STEP;
            if (k >= p.K) k = 0, first.next(p);
        }
    }
    if (!GATED) tc::grid_dependency_wait();
#pragma unroll
    for (int i = 0; i < Stages::DEPTH - 1; ++i) start(i, GATED);
    Turn<GATED> t(p);
#pragma unroll 1
    for (; t.g < s.n; t.next(p)) {
        float acc[NW][4] = {};
#pragma unroll 1
        for (int k0 = 0; k0 < p.K; k0 += STEP) {
            start(Stages::DEPTH - 1, true);
            if (AHEAD) asm volatile("cp.async.wait_group %0;" ::"n"(Stages::DEPTH - 1) : "memory");
            const int k = k0 + k_lane;
            uint4 a[NW][2];
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[i][h] = AHEAD ? ring.read(i * 2 + h) : load8<V>(row(t, i, h), k, p.K);
            const uint4 v = AHEAD ? ring.read(2 * NW) : load8<VB>(b + b_row(t), k, p.K);
#pragma unroll
            for (int i = 0; i < NW; ++i) mma_k32<BF16>(acc[i], a[i][0], a[i][1], v);
            if (!GATED) mma_k32<BF16>(acc[0], a[0][0], a[0][1], AHEAD ? ring.read(2 * NW + 1) : load8<VB>(b_lo + b_row(t), k, p.K));
            if (++ring.stage == Stages::DEPTH) ring.stage = 0;
        }
        // lane (r, c) holds weight rows r, r + 8 and rows 2c, 2c + 1 of b: red[row of b][weight row]
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[warp * NW * TILE + i * TILE + ((lane % 4) * 2 + (e & 1)) * COLS + lane / 4 + (e >> 1) * 8] = acc[i][e];
        __syncthreads();
        const int m = threadIdx.x / COLS, n = t.tile * COLS + threadIdx.x % COLS;
        if (threadIdx.x < TILE && m < s.count[t.g]) {
            float v[NW] = {};
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int w = 0; w < WARPS; ++w) v[i] += red[w * NW * TILE + i * TILE + threadIdx.x];
            if constexpr (GATED) {
                if (n < p.ldo) {  // (h is read in whole vectors: zero past N)
                    float act = 0.0f, unused;
                    with_act_device(p.act, [&](auto a) { split(act_value2<decltype(a)::value>(f2(v[0])), act, unused); });
                    const float h = n < p.N ? act * v[NW - 1] : 0.0f;
                    const T hi = from_f32<T>(h);
                    const float rest = h - to_f32(hi);
                    const int64_t at = (int64_t)s.pair[t.g][m] * p.ldo + n;
                    static_cast<T *>(p.out)[at] = hi;  // (the remainder of an infinite rounding is none)
                    static_cast<T *>(p.out_lo)[at] = from_f32<T>(isfinite(rest) ? rest : 0.0f);
                }
            } else {
                o.part[m][threadIdx.x % COLS] = v[0];
            }
        }
        if constexpr (GATED) __syncthreads();
        else add_group<T, COLS>(p, s, o, t.g);
    }
    if constexpr (!GATED) write_outputs<T, COLS>(p, o, t.tile);
}

// fp32: 4 weight rows a block, vectors of V elements.
template <int V, bool GATED>
__global__ void __launch_bounds__(THREADS, 2) expert_few_fma(const __grid_constant__ ExpertFewParams p) {
    constexpr int NW = GATED ? 2 : 1, COLS = 4, SUMS = NW * GROUP * COLS;
    __shared__ float red[WARPS][SUMS];
    __shared__ PairGroups s;
    __shared__ Outputs<GATED ? 1 : COLS> o;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    using P = Vec<float, V>;
    if (GATED) tc::grid_dependency_wait();  // (as above)
    tc::allow_dependents();
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;
    if (!GATED)
        for (int i = threadIdx.x; i < FEW_PAIRS * COLS; i += THREADS) (&o.y[0][0])[i] = 0.0f;
    sort_pairs(p, s);
    if (!GATED) tc::grid_dependency_wait();
    Turn<GATED> t(p);
#pragma unroll 1
    for (; t.g < s.n; t.next(p)) {
        const int count = s.count[t.g], n0 = t.tile * COLS;
        float acc[SUMS] = {};  // [NW][GROUP][COLS]
        const int64_t first = (int64_t)s.expert[t.g] * p.N;
        for (int k = (warp * 32 + lane) * V; k < p.K; k += THREADS * V) {
            P w[NW][COLS];
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int r = 0; r < COLS; ++r)
                    w[i][r] = *reinterpret_cast<const P *>(static_cast<const float *>(i ? p.w1 : p.w0) +
                                                           (first + min(n0 + r, p.N - 1)) * p.K + k);
#pragma unroll
            for (int m = 0; m < GROUP; ++m) {
                if (m >= count) continue;
                const int q = s.pair[t.g][m];
                const P x = *reinterpret_cast<const P *>(static_cast<const float *>(p.b) + (int64_t)(GATED ? q / p.k : q) * p.ldb + k);
#pragma unroll
                for (int i = 0; i < NW; ++i)
#pragma unroll
                    for (int r = 0; r < COLS; ++r)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            float &sum = acc[(i * GROUP + m) * COLS + r];
                            sum = fmaf(w[i][r].v[e], x.v[e], sum);
                        }
            }
        }
        const int at = fold_lanes<SUMS, 16>(acc, lane);
#pragma unroll
        for (int i = 0; i < SUMS / 32; ++i) red[warp][at + i] = acc[i];
        __syncthreads();
        const int m = threadIdx.x / COLS, n = n0 + threadIdx.x % COLS;
        if (m < count && n < p.N) {
            float v[NW] = {};
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int w = 0; w < WARPS; ++w) v[i] += red[w][i * GROUP * COLS + threadIdx.x];
            if constexpr (GATED) {
                float act = 0.0f;
                with_act_device(p.act, [&](auto a) { act = act_value<decltype(a)::value>(v[0]); });
                static_cast<float *>(p.out)[(int64_t)s.pair[t.g][m] * p.ldo + n] = act * v[NW - 1];
            } else {
                o.part[m][threadIdx.x % COLS] = v[0];
            }
        }
        if constexpr (GATED) __syncthreads();
        else add_group<float, COLS>(p, s, o, t.g);
    }
    if constexpr (!GATED) write_outputs<float, COLS>(p, o, t.tile);
}

template <auto Kernel>
cudaError_t launch(int64_t blocks, size_t smem, int cluster, cudaStream_t st, const ExpertFewParams &p) {
    const cudaError_t e = smem ? allow_smem<Kernel>((int)smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, Kernel, p);
}

template <bool GATED>
cudaError_t launch_few(ExpertFewParams &p, int dtype, cudaStream_t st) {
    const bool f32 = dtype == IM2WIN_F32, bf16 = dtype == IM2WIN_BF16;
    const int cols = f32 ? 4 : 16, pairs = p.T * p.k, most = 2 * 152;
    p.tiles = (p.N + cols - 1) / cols;
    p.shares = 1;
    int64_t blocks = p.tiles;
    if (GATED) {
        blocks = std::min<int64_t>((int64_t)p.tiles * pairs, most);  // (a pair may be a group)
    } else {
        while (p.shares < 8 && p.shares < pairs && p.tiles * p.shares * 2 <= most) p.shares *= 2;
        blocks = (int64_t)p.tiles * p.shares;
    }
    if (f32) {
        return p.K % 4 == 0 ? launch<expert_few_fma<4, GATED>>(blocks, 0, p.shares, st, p)
                            : launch<expert_few_fma<1, GATED>>(blocks, 0, p.shares, st, p);
    }
    auto go = [&](auto v, auto vb) {
        constexpr int V = decltype(v)::value, VB = decltype(vb)::value;
        const size_t smem = (V == 8 ? Ring<RING_VECS<1, GATED>>::BYTES : 0) + WARPS * (GATED ? 2 : 1) * 16 * GROUP * 4;
        return bf16 ? launch<expert_few_mma<true, V, VB, GATED>>(blocks, smem, p.shares, st, p)
                    : launch<expert_few_mma<false, V, VB, GATED>>(blocks, smem, p.shares, st, p);
    };
    // x has the weights' row length; h has rows of whole vectors
    if (p.K % 8 == 0) return go(IntC<8>(), IntC<8>());
    if (p.K % 2 == 0) return go(IntC<2>(), IntC<GATED ? 2 : 8>());
    return go(IntC<1>(), IntC<GATED ? 1 : 8>());
}

}  // namespace

cudaError_t launch_expert_few(const ExpertFew &f, int dtype, cudaStream_t st) {
    ExpertFewParams p = {};
    p.T = f.T, p.k = f.k, p.E = f.E, p.N = f.F, p.K = f.C;
    p.experts = f.experts;
    p.b = f.x, p.ldb = f.C;
    p.w0 = f.w_gate, p.w1 = f.w_up;
    p.act = f.act;
    p.out = f.h, p.out_lo = f.h_lo, p.ldo = f.ldh;
    p.status = f.status;
    const cudaError_t e = launch_few<true>(p, dtype, st);
    if (e != cudaSuccess) return e;
    ExpertFewParams q = {};
    q.T = f.T, q.k = f.k, q.E = f.E, q.N = f.C, q.K = f.F;
    q.experts = f.experts, q.weights = f.weights;
    q.b = f.h, q.b_lo = f.h_lo, q.ldb = f.ldh;
    q.w0 = f.w_down;
    q.out = f.y, q.ldo = f.C;
    return launch_few<false>(q, dtype, st);
}

}  // namespace ffn
}  // namespace im2win
