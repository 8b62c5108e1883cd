// fp32 products of the gated feed-forward on the CUDA cores: a 64 x 64 tile of D for each block of 256 threads, 4 x 4
// outputs a thread, 16 steps of K staged in shared memory as fp32.
#include "gated_ffn.cuh"

namespace im2win {
namespace ffn {
namespace {

constexpr int BM = 64, BN = 64, BK = 16, THREADS = 256, PAD = 4;

// Stages rows i0.. (64) and steps k0.. (16) of an operand as s[k][i], zero
// outside; neighbouring threads read neighbouring elements of the operand.
template <bool KMAJ>
__device__ __forceinline__ void stage(float (&s)[BK][BM + PAD], const float *p, int64_t ld, int i0, int k0, int I, int K) {
#pragma unroll
    for (int e = threadIdx.x; e < BM * BK; e += THREADS) {
        const int i = KMAJ ? e / BK : e % BM, k = KMAJ ? e % BK : e / BM;
        const bool in = i0 + i < I && k0 + k < K;
        const int64_t at = KMAJ ? (int64_t)(i0 + i) * ld + (k0 + k) : (int64_t)(k0 + k) * ld + (i0 + i);
        s[k][i] = in ? p[at] : 0.0f;
    }
}

template <bool AK, bool BKM, int EPI, int ACT>
__global__ void __launch_bounds__(THREADS) simt_product(Product p, int tiles_n) {
    constexpr int NB = EPI == EPI_GATED ? 2 : 1;  // accumulators
    __shared__ float sa[BK][BM + PAD], sb[NB][BK][BN + PAD];
    const int m0 = (int)(blockIdx.x / tiles_n) * BM, n0 = (int)(blockIdx.x % tiles_n) * BN;
    const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
    float acc[NB][4][4] = {};
    const int segs = EPI != EPI_GATED && p.a1.p ? 2 : 1;
    for (int seg = 0; seg < segs; ++seg) {
        const float *a = static_cast<const float *>(seg ? p.a1.p : p.a0.p);
        const float *b = static_cast<const float *>(seg ? p.b1.p : p.b0.p);
        for (int k0 = 0; k0 < p.K; k0 += BK) {
            stage<AK>(sa, a, p.a0.ld, m0, k0, p.M, p.K);
            stage<BKM>(sb[0], b, p.b0.ld, n0, k0, p.N, p.K);
            if (NB == 2) stage<BKM>(sb[NB - 1], static_cast<const float *>(p.b1.p), p.b1.ld, n0, k0, p.N, p.K);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < BK; ++k) {
                float av[4], bv[NB][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) av[i] = sa[k][tm + i];
#pragma unroll
                for (int q = 0; q < NB; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) bv[q][j] = sb[q][k][tn + j];
#pragma unroll
                for (int q = 0; q < NB; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[q][i][j] = fmaf(av[i], bv[q][j], acc[q][i][j]);
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + tm + i, n = n0 + tn + j;
            if (m >= p.M || n >= p.N) continue;
            float *out = static_cast<float *>(p.out) + (int64_t)m * p.ldo + n;
            const int64_t at = kept_index(m, n, p.N);
            if (EPI == EPI_STORE) {
                *out = acc[0][i][j];
            } else if (EPI == EPI_GATED) {
                const float g = acc[0][i][j], u = acc[NB - 1][i][j];
                *out = act_value<ACT>(g) * u;
                if (p.g) p.g[at] = g, p.u[at] = u;
            } else {
                float a, d;
                act_both<ACT>(p.g[at], a, d);
                *out = acc[0][i][j] * p.u[at] * d;
                static_cast<float *>(p.out2)[(int64_t)m * p.ldo + n] = acc[0][i][j] * a;
            }
        }
}

template <bool AK, bool BKM, int EPI, int ACT>
cudaError_t launch(const Product &p, cudaStream_t st) {
    const int64_t tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
    if (tm * tn > 0x7fffffff) return cudaErrorInvalidValue;
    simt_product<AK, BKM, EPI, ACT><<<(unsigned)(tm * tn), THREADS, 0, st>>>(p, (int)tn);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_simt(const Product &p, cudaStream_t st) {
    cudaError_t e = cudaErrorInvalidValue;
    if (p.epi == EPI_GATED)
        with_act(p.act, [&](auto a) { e = launch<true, true, EPI_GATED, decltype(a)::value>(p, st); });
    else if (p.epi == EPI_DGATED)
        with_act(p.act, [&](auto a) { e = launch<true, false, EPI_DGATED, decltype(a)::value>(p, st); });
    else if (p.a0.k_major)
        e = p.b0.k_major ? launch<true, true, EPI_STORE, 0>(p, st) : launch<true, false, EPI_STORE, 0>(p, st);
    else
        e = launch<false, false, EPI_STORE, 0>(p, st);
    return e;
}

}  // namespace ffn
}  // namespace im2win
