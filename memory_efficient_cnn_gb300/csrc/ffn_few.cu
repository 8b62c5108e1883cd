// Gated feed-forward of few rows, bound by reading the weights once.
//
// fp16/bf16: a warp multiplies 16 weight rows with up to 32 rows of x by
// mma.sync, whose operands need no exchange between lanes: the order of
// the summed index is free as long as both operands agree, so lane (r, c) takes
// the 8 consecutive elements 8c.. of its row as the fragments of two steps, one
// 16-byte load each. (A tcgen05 product would stage 128 rows for these few and
// join split sums by a second kernel; the tensor rate needed here is below one
// percent of either path.) The 8 warps of a block split the summed index and are
// joined in order. h goes to the second product as its rounding and the
// remainder of that, two 16-bit numbers, at the cost of a second MMA a step: it
// keeps 16 bits of bf16's 8 and 22 of fp16's 11.
//
// fp32: the same split on the CUDA cores, 4 weight rows a block and up to 8 rows of x;
// more rows take more blocks, which find the weights in L2.
//
// Measured with blocks of weights of 4096 x 10240, 252 MB in bf16: 43 us for one row
// and 47 us for five, 5.9 and 5.4 TB/s; 58 us for sixteen. fp32, 4096 x 8192, 403 MB:
// 60 us for one row (6.7 TB/s: memory), 69 us for four, 102 us for eight, whose loads
// of x count for more than the weights'.
#include <algorithm>

#include "gated_ffn.cuh"
#include "tc_ptx.cuh"

namespace im2win {
namespace ffn {
namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;

struct FewParams {
    int R, N, K;               // rows; weight rows; summed index
    const void *b, *b_lo;      // [R][ldb]: x, or h and its remainder
    int64_t ldb;
    const void *w0, *w1;       // [N][K]; gate and up, or down alone
    int act;
    void *out, *out_lo;        // h and its remainder, or y
    int64_t ldo;
    void *kept;                // act(g) and u act'(g), where not null
    uint16_t *planes;          // fp32: h in planes too then
    int64_t plane_ld;
    uint32_t *status;          // cleared where not null
};

// 8 elements from p[k] on, zero past K; vectors of V elements are aligned and whole.
template <int V>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int k, int K) {
    if (V == 8) return k < K ? *reinterpret_cast<const uint4 *>(p + k) : make_uint4(0, 0, 0, 0);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (V == 2) {
            v[i] = k + 2 * i < K ? *reinterpret_cast<const uint32_t *>(p + k + 2 * i) : 0u;
        } else {
            const uint32_t lo = k + 2 * i < K ? p[k + 2 * i] : 0u, hi = k + 2 * i + 1 < K ? p[k + 2 * i + 1] : 0u;
            v[i] = lo | (hi << 16);
        }
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 steps of the summed index: 16 weight rows (two loads) by 8 rows of b.
template <bool BF16>
__device__ __forceinline__ void mma_k32(float (&d)[4], const uint4 &top, const uint4 &bottom, const uint4 &b) {
    mma16816<BF16>(d, top.x, bottom.x, top.y, bottom.y, b.x, b.y);
    mma16816<BF16>(d, top.z, bottom.z, top.w, bottom.w, b.z, b.w);
}

// What a lane will multiply, on its way: it copies ahead itself, so that its part
// of a block's stages needs no barrier. A stage is 32 steps of the summed index:
// VECS vectors a lane. b goes through it too: it comes from L2, whose answers
// take longer than a stage when the weights keep the memory busy.
template <int VECS>
struct Ring {
    static constexpr int DEPTH = 96 * 1024 / (VECS * 16 * THREADS) < 2 ? 2 : 96 * 1024 / (VECS * 16 * THREADS);
    static constexpr int BYTES = DEPTH * VECS * 16 * THREADS;
    uint32_t base;
    int stage = 0;
    __device__ explicit Ring(const void *smem) : base((uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16) {}
    __device__ __forceinline__ uint32_t at(int s, int v) const { return base + (s * VECS + v) * (16 * THREADS); }
    __device__ __forceinline__ void copy(int ahead, int v, const uint16_t *src, bool in) {
        int s = stage + ahead;
        if (s >= DEPTH) s -= DEPTH;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(s, v)), "l"(src), "r"(in ? 16 : 0) : "memory");
    }
    __device__ __forceinline__ uint4 read(int v) const {
        uint4 r;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "r"(at(stage, v))
                     : "memory");
        return r;
    }
};
template <int NT, bool GATED>
constexpr int RING_VECS = GATED ? 4 + NT : 2 + 2 * NT;

// NT: groups of 8 rows of b. V, VB: vectors of the weights and of b. A block takes
// tiles of 16 weight rows in turn; with whole vectors the next stages' copies go
// on over the ends of tiles.
template <bool BF16, int NT, int V, int VB, bool GATED>
__global__ void __launch_bounds__(THREADS, NT <= 2 ? 2 : 1) few_mma(const __grid_constant__ FewParams p, int tiles) {
    using T = std::conditional_t<BF16, bf16_t, f16_t>;
    constexpr int NW = GATED ? 2 : 1;   // weight matrices
    constexpr int TILE = 16 * 8 * NT;   // sums of one of them
    constexpr int STEP = WARPS * 32;    // of the summed index, of a block
    constexpr bool AHEAD = V == 8;
    using Stages = Ring<RING_VECS<NT, GATED>>;
    extern __shared__ uint4 dyn[];
    float *red = reinterpret_cast<float *>(dyn) + (AHEAD ? Stages::BYTES / 4 : 0);  // [WARPS][NW * TILE]
    Stages ring(dyn);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k_lane = warp * 32 + (lane % 4) * 8;
    const uint16_t *b[NT], *bl[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t off = (int64_t)min(t * 8 + lane / 4, p.R - 1) * p.ldb;
        b[t] = static_cast<const uint16_t *>(p.b) + off;
        bl[t] = GATED ? nullptr : static_cast<const uint16_t *>(p.b_lo) + off;
    }
    // weight row h (0, 1: eight rows apart) of the lane in matrix i, of tile n
    auto row = [&](int n, int i, int h) {
        return static_cast<const uint16_t *>(i ? p.w1 : p.w0) + (int64_t)min(n * 16 + lane / 4 + h * 8, p.N - 1) * p.K;
    };
    int next_tile = blockIdx.x, next_k = 0;  // of the copies
    auto copy_weights = [&](int ahead, int tile, int k) {
        const bool in = k < p.K;
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) ring.copy(ahead, i * 2 + h, row(tile, i, h) + (in ? k : 0), in);
    };
    auto start = [&](int ahead, bool weights) {
        if (!AHEAD) return;
        if (next_tile < tiles) {
            const int k = next_k + k_lane;
            const bool in = k < p.K;
            const int64_t at = in ? k : 0;
            if (weights) copy_weights(ahead, next_tile, k);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                // (a row that is not there is not read: one line asked for by every warp costs L2 more
                // than the weights)
                const bool there = in && t * 8 + lane / 4 < p.R;
                ring.copy(ahead, 2 * NW + t, b[t] + at, there);
                if (!GATED) ring.copy(ahead, 2 * NW + NT + t, bl[t] + at, there);
            }
            next_k += STEP;
            if (next_k >= p.K) next_k = 0, next_tile += gridDim.x;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // The second launch begins while the first runs, which has waited for all before it and
    // writes h alone: the first weights need not wait for it.
    if (AHEAD && !GATED) {
        int tile = blockIdx.x, k = 0;
#pragma unroll
        for (int s = 0; s < Stages::DEPTH - 1; ++s) {
            if (tile < tiles) copy_weights(s, tile, k + k_lane);
            k += STEP;
            if (k >= p.K) k = 0, tile += gridDim.x;
        }
    }
    tc::grid_dependency_wait();
    tc::allow_dependents();
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;
#pragma unroll
    for (int s = 0; s < Stages::DEPTH - 1; ++s) start(s, GATED);

#pragma unroll 1
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        float acc[NW][NT][4] = {};
#pragma unroll 1
        for (int k0 = 0; k0 < p.K; k0 += STEP) {
            start(Stages::DEPTH - 1, true);
            if (AHEAD) asm volatile("cp.async.wait_group %0;" ::"n"(Stages::DEPTH - 1) : "memory");
            const int k = k0 + k_lane;
            uint4 a[NW][2];
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[i][h] = AHEAD ? ring.read(i * 2 + h) : load8<V>(row(tile, i, h), k, p.K);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint4 v = AHEAD ? ring.read(2 * NW + t) : load8<VB>(b[t], k, p.K);
#pragma unroll
                for (int i = 0; i < NW; ++i) mma_k32<BF16>(acc[i][t], a[i][0], a[i][1], v);
                if (!GATED)
                    mma_k32<BF16>(acc[0][t], a[0][0], a[0][1], AHEAD ? ring.read(2 * NW + NT + t) : load8<VB>(bl[t], k, p.K));
            }
            if (++ring.stage == Stages::DEPTH) ring.stage = 0;
        }
        // lane (r, c) holds weight rows r, r + 8 and rows 2c, 2c + 1 of b: red[row of b][weight row]
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    red[warp * NW * TILE + i * TILE + (t * 8 + (lane % 4) * 2 + (e & 1)) * 16 + lane / 4 + (e >> 1) * 8] =
                        acc[i][t][e];
        __syncthreads();
        for (int e = threadIdx.x; e < TILE; e += THREADS) {
            const int m = e / 16, n = tile * 16 + e % 16;
            if (m >= p.R) continue;
            if (n >= p.N) {
                if (GATED && n < p.ldo) {  // h is read in whole vectors
                    static_cast<T *>(p.out)[(int64_t)m * p.ldo + n] = from_f32<T>(0.0f);
                    static_cast<T *>(p.out_lo)[(int64_t)m * p.ldo + n] = from_f32<T>(0.0f);
                }
                continue;
            }
            float v[NW] = {};
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int k = 0; k < WARPS; ++k) v[i] += red[k * NW * TILE + i * TILE + e];
            T *out = static_cast<T *>(p.out) + (int64_t)m * p.ldo + n;
            if (GATED) {
                float act = 0.0f, slope = 0.0f, unused;
                with_act_device(p.act, [&](auto a) {
                    F2 x, y;
                    act_both2<decltype(a)::value>(f2(v[0]), x, y);
                    split(x, act, unused);
                    split(y, slope, unused);
                });
                const float h = act * v[NW - 1];
                const T hi = from_f32<T>(h);
                const float rest = h - to_f32(hi);
                *out = hi;  // (the remainder of an infinite rounding is none)
                static_cast<T *>(p.out_lo)[(int64_t)m * p.ldo + n] = from_f32<T>(isfinite(rest) ? rest : 0.0f);
                if (p.kept) {
                    unsigned char *at = static_cast<unsigned char *>(p.kept) + kept_block(m, n, p.N);
                    const float keep[2] = {act, slope * v[NW - 1]};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t bits = __float_as_uint(keep[i]);
                        *reinterpret_cast<uint16_t *>(at + i * 512 + n % 8 * 2) = (uint16_t)(bits >> 16);
                        at[1024 + i * 8 + n % 8] = (unsigned char)(bits >> 8);
                    }
                }
            } else {
                *out = from_f32<T>(v[0]);
            }
        }
        __syncthreads();
    }
}

// Sums of N values over a warp's lanes. While there are two or more, a lane hands
// half of them to its partner and goes on with the other half; it ends with those
// from the returned index on (butterflies of all N: 150 us instead of 132 us for
// eight rows of 4096 x 8192).
template <int N, int O, int SIZE>
__device__ __forceinline__ int fold_lanes(float (&v)[SIZE], int lane) {
    if constexpr (O == 0) {
        return 0;
    } else if constexpr (N == 1) {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
        return fold_lanes<1, O / 2>(v, lane);
    } else {
        const bool upper = (lane & O) != 0;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = upper ? v[i + N / 2] : v[i], give = upper ? v[i] : v[i + N / 2];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, O);
        }
        return (upper ? N / 2 : 0) + fold_lanes<N / 2, O / 2>(v, lane);
    }
}

// fp32: NR rows of b and 4 weight rows a block, vectors of V elements. From four rows
// on two blocks an SM, of one step at a time (one block of two steps: 132 us instead
// of 102 us for eight rows of 4096 x 8192); below, registers for two steps in flight.
template <int NR, int V, bool GATED>
__global__ void __launch_bounds__(THREADS, NR >= 4 ? 2 : 1) few_fma(const __grid_constant__ FewParams p) {
    constexpr int NW = GATED ? 2 : 1, ROWS = 4, SUMS = NW * ROWS * NR;
    __shared__ float red[WARPS][SUMS];
    // blocks of the same weights and other rows follow one another, so that L2 has the weights
    const int groups = (p.R + NR - 1) / NR, m0 = blockIdx.x % groups * NR, n0 = blockIdx.x / groups * ROWS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    using P = Vec<float, V>;
    float acc[SUMS] = {};  // [NW][NR][ROWS]
    tc::grid_dependency_wait();
    tc::allow_dependents();
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;
#pragma unroll (NR * NW <= 4 ? 2 : 1)
    for (int k = (warp * 32 + lane) * V; k < p.K; k += THREADS * V) {
        P w[NW][ROWS];
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                w[i][r] = *reinterpret_cast<const P *>(static_cast<const float *>(i ? p.w1 : p.w0) +
                                                       (int64_t)min(n0 + r, p.N - 1) * p.K + k);
#pragma unroll
        for (int m = 0; m < NR; ++m) {
            const P x = *reinterpret_cast<const P *>(static_cast<const float *>(p.b) + (int64_t)min(m0 + m, p.R - 1) * p.ldb + k);
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float &sum = acc[(i * NR + m) * ROWS + r];
                        sum = fmaf(w[i][r].v[e], x.v[e], sum);
                    }
        }
    }
    const int first = fold_lanes<SUMS, 16>(acc, lane);
    if (SUMS >= 32 || lane % (32 / SUMS) == 0) {
#pragma unroll
        for (int i = 0; i < (SUMS + 31) / 32; ++i) red[warp][first + i] = acc[i];
    }
    __syncthreads();
    if (threadIdx.x >= NR * ROWS) return;
    const int m = m0 + threadIdx.x / ROWS, n = n0 + threadIdx.x % ROWS;
    if (m >= p.R || n >= p.N) return;
    float v[NW] = {};
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int k = 0; k < WARPS; ++k) v[i] += red[k][i * NR * ROWS + threadIdx.x];
    float *out = static_cast<float *>(p.out) + (int64_t)m * p.ldo + n;
    if (GATED) {
        float act = 0.0f, slope = 0.0f;
        with_act_device(p.act, [&](auto a) { act_both<decltype(a)::value>(v[0], act, slope); });
        const float h = act * v[NW - 1];
        *out = h;
        if (p.kept) {
            float *at = static_cast<float *>(p.kept) + kept_index_f32(m, n, p.N);
            at[0] = act, at[kept_count_f32(p.R, p.N)] = slope * v[NW - 1];
            uint16_t *plane = p.planes + (int64_t)m * p.plane_ld + n;
            const int64_t next = p.R * p.plane_ld;
            split_f32(h, plane[0], plane[next], plane[2 * next]);
        }
    } else {
        *out = v[0];
    }
}

template <typename K, typename... A>
cudaError_t launch(K kernel, int blocks, size_t smem, cudaStream_t st, A... args) {
    if (smem) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool BF16, int NT, int V, int VB, bool GATED>
cudaError_t launch_tiles(const FewParams &p, cudaStream_t st) {
    constexpr int NW = GATED ? 2 : 1;
    const size_t smem = (V == 8 ? Ring<RING_VECS<NT, GATED>>::BYTES : 0) + WARPS * NW * 16 * 8 * NT * 4;
    // as many blocks as fit at a time, or fewer that all take the same number of tiles
    const int tiles = (p.N + 15) / 16, most = 152 * (NT <= 2 ? 2 : 1), rounds = (tiles + most - 1) / most;
    return launch(few_mma<BF16, NT, V, VB, GATED>, (tiles + rounds - 1) / rounds, smem, st, p, tiles);
}

template <bool BF16, int NT, bool GATED>
cudaError_t launch_mma(const FewParams &p, cudaStream_t st) {
    // x has the weights' row length; h has rows of whole vectors
    if (p.K % 8 == 0) return launch_tiles<BF16, NT, 8, 8, GATED>(p, st);
    if (p.K % 2 == 0) return launch_tiles<BF16, NT, 2, GATED ? 2 : 8, GATED>(p, st);
    return launch_tiles<BF16, NT, 1, GATED ? 1 : 8, GATED>(p, st);
}

template <bool BF16, bool GATED>
cudaError_t launch_16(const FewParams &p, cudaStream_t st) {
    if (p.R <= 8) return launch_mma<BF16, 1, GATED>(p, st);
    if (p.R <= 16) return launch_mma<BF16, 2, GATED>(p, st);
    return launch_mma<BF16, 4, GATED>(p, st);
}

template <int NR, bool GATED>
cudaError_t launch_fma(const FewParams &p, cudaStream_t st) {
    const int blocks = (p.N + 3) / 4 * ((p.R + NR - 1) / NR);
    return p.K % 4 == 0 ? launch(few_fma<NR, 4, GATED>, blocks, 0, st, p) : launch(few_fma<NR, 1, GATED>, blocks, 0, st, p);
}

template <bool GATED>
cudaError_t launch_32(const FewParams &p, cudaStream_t st) {
    if (p.R <= 1) return launch_fma<1, GATED>(p, st);
    if (p.R <= 2) return launch_fma<2, GATED>(p, st);
    if (p.R <= 4) return launch_fma<4, GATED>(p, st);
    return launch_fma<8, GATED>(p, st);
}

template <bool GATED>
cudaError_t launch_any(const FewParams &p, int dtype, cudaStream_t st) {
    if (dtype == IM2WIN_F32) return launch_32<GATED>(p, st);
    return dtype == IM2WIN_BF16 ? launch_16<true, GATED>(p, st) : launch_16<false, GATED>(p, st);
}

}  // namespace

// Where these kernels are the faster ones. 16-bit types: up to 16 rows (1024 x 4096:
// 13 us against 19 us of the tensor-memory products; 4096 x 10240: 58 us against 57
// us); up to 32 rows for small weights, where the products' partial sums count for
// more than the second reading of b here (32 rows of 512 x 1536: 8 us against 14 us;
// 2048 x 4096: 26 us against 28 us; 2048 x 8192: 46 us against 31 us). fp32: up to 32
// rows (2048 x 4096: 48 us against 90 us for 16 rows, 87 us against 92 us for 32), and
// up to 128 where the work is small (64 rows of 256 x 640: 13 us against 25 us; of 384 x
// 1001: 22 us against 29 us; of 1024 x 2816: 76 us against 43 us).
bool is_few(int64_t R, int64_t C, int64_t F, int dtype) {
    if (dtype == IM2WIN_F32) return R <= 32 || (R <= 128 && R * C * F <= (int64_t(1) << 24));
    return R <= 16 || (R <= 32 && C * F <= (int64_t(8) << 20));
}

cudaError_t launch_few(const Few &f, int dtype, cudaStream_t st) {
    FewParams p = {};
    p.R = f.R; p.N = f.F; p.K = f.C;
    p.b = f.x; p.ldb = f.C;
    p.w0 = f.w_gate; p.w1 = f.w_up;
    p.act = f.act;
    p.out = f.h; p.out_lo = f.h_lo; p.ldo = f.ldh;
    p.kept = f.kept;
    p.planes = f.planes; p.plane_ld = f.plane_ld;
    p.status = f.status;
    const cudaError_t e = launch_any<true>(p, dtype, st);
    if (e != cudaSuccess) return e;
    FewParams q = {};
    q.R = f.R; q.N = f.C; q.K = f.F;
    q.b = f.h; q.b_lo = f.h_lo; q.ldb = f.ldh;
    q.w0 = f.w_down;
    q.out = f.y; q.ldo = f.C;
    return launch_any<false>(q, dtype, st);
}

}  // namespace ffn
}  // namespace im2win
