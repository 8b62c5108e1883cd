// Gated feed-forward of few rows, bound by reading the weights once.
//
// fp16/bf16: a warp multiplies 16 weight rows with up to 32 rows of x by
// mma.sync, whose operands go from memory straight to registers: the order of
// the summed index is free as long as both operands agree, so lane (r, c) takes
// the 8 consecutive elements 8c.. of its row as the fragments of two steps, one
// 16-byte load each. (A tcgen05 product would stage 128 rows for these few and
// join split sums by a second kernel; the tensor rate needed here is below one
// percent of either path.) The 8 warps of a block split the summed index and are
// joined in order. h goes to the second product as its rounding and the
// remainder of that, two 16-bit numbers, at the cost of a second MMA a step: it
// keeps 16 bits of bf16's 8 and 22 of fp16's 11.
//
// fp32: the same split on the CUDA cores, 4 weight rows a warp.
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
    float *g, *u;              // kept in fp32 where not null
    uint32_t *status;          // cleared where not null
};

// 8 elements from p[k] on, zero past K; vectors of V elements are aligned and whole.
template <int V>
__device__ __forceinline__ uint4 load8(const uint16_t *p, int k, int K, bool cached) {
    if (V == 8) {
        if (k >= K) return make_uint4(0, 0, 0, 0);
        return cached ? *reinterpret_cast<const uint4 *>(p + k) : __ldcs(reinterpret_cast<const uint4 *>(p + k));
    }
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

// NT: groups of 8 rows of b. V, VB: vectors of the weights and of b.
template <bool BF16, int NT, int V, int VB, bool GATED>
__global__ void __launch_bounds__(THREADS) few_mma(const __grid_constant__ FewParams p) {
    using T = std::conditional_t<BF16, bf16_t, f16_t>;
    constexpr int NW = GATED ? 2 : 1;   // weight matrices
    constexpr int TILE = 16 * 8 * NT;   // sums of one of them
    __shared__ float red[WARPS][NW * TILE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * 16;
    const int r0 = min(n0 + lane / 4, p.N - 1), r1 = min(n0 + lane / 4 + 8, p.N - 1);
    const uint16_t *w[NW][2], *b[NT], *bl[NT];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const uint16_t *base = static_cast<const uint16_t *>(i ? p.w1 : p.w0);
        w[i][0] = base + (int64_t)r0 * p.K;
        w[i][1] = base + (int64_t)r1 * p.K;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t off = (int64_t)min(t * 8 + lane / 4, p.R - 1) * p.ldb;
        b[t] = static_cast<const uint16_t *>(p.b) + off;
        bl[t] = GATED ? nullptr : static_cast<const uint16_t *>(p.b_lo) + off;
    }
    float acc[NW][NT][4] = {};
    tc::grid_dependency_wait();
    tc::allow_dependents();
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;

    constexpr int STEPS = NT <= 2 ? 4 : 2;  // of 32, in flight together
#pragma unroll 1
    for (int k0 = warp * 32 * STEPS; k0 < p.K; k0 += WARPS * 32 * STEPS) {
        uint4 a[STEPS][NW][2];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[s][i][h] = load8<V>(w[i][h], k0 + s * 32 + (lane % 4) * 8, p.K, false);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + s * 32 + (lane % 4) * 8;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint4 v = load8<VB>(b[t], k, p.K, true);
#pragma unroll
                for (int i = 0; i < NW; ++i) mma_k32<BF16>(acc[i][t], a[s][i][0], a[s][i][1], v);
                if (!GATED) mma_k32<BF16>(acc[0][t], a[s][0][0], a[s][0][1], load8<VB>(bl[t], k, p.K, true));
            }
        }
    }
    // lane (r, c) holds weight rows r, r + 8 and rows 2c, 2c + 1 of b: red[row of b][weight row]
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[warp][i * TILE + (t * 8 + (lane % 4) * 2 + (e & 1)) * 16 + lane / 4 + (e >> 1) * 8] = acc[i][t][e];
    __syncthreads();
    for (int e = threadIdx.x; e < TILE; e += THREADS) {
        const int m = e / 16, n = n0 + e % 16;
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
            for (int k = 0; k < WARPS; ++k) v[i] += red[k][i * TILE + e];
        T *out = static_cast<T *>(p.out) + (int64_t)m * p.ldo + n;
        if (GATED) {
            float h = 0.0f;
            with_act_device(p.act, [&](auto a) {
                float unused;
                split(act_value2<decltype(a)::value>(f2(v[0])), h, unused);
            });
            h *= v[NW - 1];
            const T hi = from_f32<T>(h);
            const float rest = h - to_f32(hi);
            *out = hi;  // (the remainder of an infinite rounding is none)
            static_cast<T *>(p.out_lo)[(int64_t)m * p.ldo + n] = from_f32<T>(isfinite(rest) ? rest : 0.0f);
            if (p.g) p.g[kept_index(m, n, p.N)] = v[0], p.u[kept_index(m, n, p.N)] = v[NW - 1];
        } else {
            *out = from_f32<T>(v[0]);
        }
    }
}

// fp32: NR rows of b, 4 weight rows a block, vectors of V elements.
template <int NR, int V, bool GATED>
__global__ void __launch_bounds__(THREADS) few_fma(const __grid_constant__ FewParams p) {
    constexpr int NW = GATED ? 2 : 1, ROWS = 4, SUMS = NW * ROWS * NR;
    __shared__ float red[WARPS][SUMS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n0 = blockIdx.x * ROWS;
    using P = Vec<float, V>;
    float acc[NW][ROWS][NR] = {};
    tc::grid_dependency_wait();
    tc::allow_dependents();
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;
#pragma unroll 2
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
            const P x = *reinterpret_cast<const P *>(static_cast<const float *>(p.b) + (int64_t)min(m, p.R - 1) * p.ldb + k);
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[i][r][m] = fmaf(w[i][r].v[e], x.v[e], acc[i][r][m]);
        }
    }
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int m = 0; m < NR; ++m) {
                float v = acc[i][r][m];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0) red[warp][(i * NR + m) * ROWS + r] = v;
            }
    __syncthreads();
    if (threadIdx.x >= NR * ROWS) return;
    const int m = threadIdx.x / ROWS, n = n0 + threadIdx.x % ROWS;
    if (m >= p.R || n >= p.N) return;
    float v[NW] = {};
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int k = 0; k < WARPS; ++k) v[i] += red[k][i * NR * ROWS + threadIdx.x];
    float *out = static_cast<float *>(p.out) + (int64_t)m * p.ldo + n;
    if (GATED) {
        float h = 0.0f;
        with_act_device(p.act, [&](auto a) { h = act_value<decltype(a)::value>(v[0]) * v[NW - 1]; });
        *out = h;
        if (p.g) p.g[kept_index(m, n, p.N)] = v[0], p.u[kept_index(m, n, p.N)] = v[NW - 1];
    } else {
        *out = v[0];
    }
}

template <typename K>
cudaError_t launch(K kernel, int blocks, const FewParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool BF16, int NT, bool GATED>
cudaError_t launch_mma(const FewParams &p, cudaStream_t st) {
    const int blocks = (p.N + 15) / 16;
    // x has the weights' row length; h has rows of whole vectors
    if (p.K % 8 == 0) return launch(few_mma<BF16, NT, 8, 8, GATED>, blocks, p, st);
    if (p.K % 2 == 0) return launch(few_mma<BF16, NT, 2, GATED ? 2 : 8, GATED>, blocks, p, st);
    return launch(few_mma<BF16, NT, 1, GATED ? 1 : 8, GATED>, blocks, p, st);
}

template <bool BF16, bool GATED>
cudaError_t launch_16(const FewParams &p, cudaStream_t st) {
    if (p.R <= 8) return launch_mma<BF16, 1, GATED>(p, st);
    if (p.R <= 16) return launch_mma<BF16, 2, GATED>(p, st);
    return launch_mma<BF16, 4, GATED>(p, st);
}

template <int NR, bool GATED>
cudaError_t launch_fma(const FewParams &p, cudaStream_t st) {
    const int blocks = (p.N + 3) / 4;
    return p.K % 4 == 0 ? launch(few_fma<NR, 4, GATED>, blocks, p, st) : launch(few_fma<NR, 1, GATED>, blocks, p, st);
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

int few_rows(int dtype) { return dtype == IM2WIN_F32 ? 8 : 32; }

cudaError_t launch_few(const Few &f, int dtype, cudaStream_t st) {
    FewParams p = {};
    p.R = f.R; p.N = f.F; p.K = f.C;
    p.b = f.x; p.ldb = f.C;
    p.w0 = f.w_gate; p.w1 = f.w_up;
    p.act = f.act;
    p.out = f.h; p.out_lo = f.h_lo; p.ldo = f.ldh;
    p.g = f.g; p.u = f.u;
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
