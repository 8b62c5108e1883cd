// fp32 products of the gated feed-forward on the CUDA cores.
//
// A 128 x 64 tile of D (EPI_GATED: 32 columns of g and the same of u) for each
// block of 256 threads: two groups of 128, each with half of the K blocks and
// 8 x 8 outputs a thread, so that outputs of as few tiles as there are SMs still
// have two warps on each scheduler; the groups' sums are added at the end. The
// operands' elements are copied asynchronously to shared memory with K outermost,
// three blocks of 16 K steps in flight, from either layout and any alignment.
// The inner product is on pairs of columns (paired fp32 FMAs: half the issue
// slots, which leaves room for the shared-memory reads).
#include "gated_ffn.cuh"
#include "tc_ptx.cuh"

namespace im2win {
namespace ffn {
namespace {

constexpr int BM = 128, BN = 64, BK = 16, GROUP = 128, GROUPS = 2, THREADS = GROUP * GROUPS, STAGES = 3;
constexpr int PITCH_A = BM + 4, PITCH_B = BN + 4;    // floats; 16-byte aligned rows
constexpr int STAGE = BK * (PITCH_A + PITCH_B);      // floats
constexpr int SMEM = GROUPS * STAGES * STAGE * 4;
static_assert(SMEM >= GROUPS * 32 * GROUP * 8, "the sums at the end take the stages' place");

__device__ __forceinline__ void copy4(float *dst, const float *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(in ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy16(float *dst, const float *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(bytes)
                 : "memory");
}

// Starts copying output indexes i0.. (N of them) and K steps k0.. (16) of an operand
// to s[k][i], zero outside; neighbouring threads copy neighbouring elements, four
// at a time where the output index is innermost and rows are 16-byte aligned.
template <bool KMAJ, int N, int PITCH>
__device__ __forceinline__ void stage(float *s, const float *p, int64_t ld, int i0, int k0, int I, int K, int t) {
    if (!KMAJ && (ld & 3) == 0) {
#pragma unroll
        for (int e = 0; e < N * BK / (4 * GROUP); ++e) {
            const int x = e * GROUP + t, i = x % (N / 4) * 4, k = x / (N / 4);
            const int left = k0 + k < K ? min(I - i0 - i, 4) : 0;
            copy16(s + k * PITCH + i, left > 0 ? p + (int64_t)(k0 + k) * ld + (i0 + i) : p, left > 0 ? 4 * left : 0);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < N * BK / GROUP; ++e) {
        const int x = e * GROUP + t;
        // (K innermost: 8 steps of 4 output indexes a warp, whose words fall in 32 banks)
        const int i = KMAJ ? x / 8 % N : x % N, k = KMAJ ? x % 8 + x / (8 * N) * 8 : x / N;
        const bool in = i0 + i < I && k0 + k < K;
        const int64_t at = KMAJ ? (int64_t)(i0 + i) * ld + (k0 + k) : (int64_t)(k0 + k) * ld + (i0 + i);
        copy4(s + k * PITCH + i, in ? p + at : p, in);
    }
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at `p` in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ uint64_t load_of_rank(const uint64_t *p, int rank) {
    uint32_t a;
    uint64_t v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

template <bool AK, bool BKM, int EPI, int ACT>
__global__ void __launch_bounds__(THREADS, 2) simt_product(const __grid_constant__ Product p, int tiles_n, int tiles, int share) {
    extern __shared__ uint4 dyn[];
    constexpr bool GATED = EPI == EPI_GATED;
    constexpr int COLS = GATED ? BN / 2 : BN;
    const int rank = (int)blockIdx.x % share, id = (int)blockIdx.x / share;
    const int z = p.batch ? id / tiles : 0, tile = id - z * tiles;
    const int m0 = tile / tiles_n * BM, n0 = tile % tiles_n * COLS;
    const int group = threadIdx.x / GROUP, t = threadIdx.x % GROUP;
    float *mine = reinterpret_cast<float *>(dyn) + group * STAGES * STAGE;
    // the thread's rows r0.., r0 + 64.. and columns c0.., c0 + 32.. (of g and of u), four each:
    // a warp's reads of a stage are contiguous
    const int r0 = t / 8 * 4, c0 = t % 8 * 4;
    const int segs = !GATED && !p.batch && p.a1.p ? 2 : 1;
    const int KB = (p.K + BK - 1) / BK, total = KB * segs;

    // the group's K blocks: `first`, `first` + step, ...
    const int first = rank * GROUPS + group, step = GROUPS * share;
    auto start = [&](int j) {  // the group's j-th
        const int b = first + j * step;
        if (b < total) {
            const int seg = b >= KB ? 1 : 0, k0 = (b - seg * KB) * BK;
            float *sa = mine + j % STAGES * STAGE, *sb = sa + BK * PITCH_A;
            stage<AK, BM, PITCH_A>(sa, static_cast<const float *>(seg || z ? p.a1.p : p.a0.p), p.a0.ld, m0, k0, p.M, p.K, t);
            if (GATED) {
                stage<BKM, COLS, PITCH_B>(sb, static_cast<const float *>(p.b0.p), p.b0.ld, n0, k0, p.N, p.K, t);
                stage<BKM, COLS, PITCH_B>(sb + COLS, static_cast<const float *>(p.b1.p), p.b0.ld, n0, k0, p.N, p.K, t);
            } else {
                stage<BKM, BN, PITCH_B>(sb, static_cast<const float *>(seg || z ? p.b1.p : p.b0.p), p.b0.ld, n0, k0, p.N, p.K, t);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    F2 acc[4][8];  // [pair of rows][column]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = f2(0.0f);
    start(0);
    start(1);
#pragma unroll 1
    for (int j = 0; first + j * step < total; ++j) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        // every thread's copies of this block have landed, and every thread is done with the
        // block before it, whose stage the next copies take
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(GROUP) : "memory");
        start(j + 2);
        const float *sa = mine + j % STAGES * STAGE, *sb = sa + BK * PITCH_A;
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const ulonglong2 lo = *reinterpret_cast<const ulonglong2 *>(sa + k * PITCH_A + r0);
            const ulonglong2 hi = *reinterpret_cast<const ulonglong2 *>(sa + k * PITCH_A + r0 + 64);
            const float4 b0 = *reinterpret_cast<const float4 *>(sb + k * PITCH_B + c0);
            const float4 b1 = *reinterpret_cast<const float4 *>(sb + k * PITCH_B + c0 + 32);
            const F2 a[4] = {{lo.x}, {lo.y}, {hi.x}, {hi.y}};
            const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][n] = fma2(a[i], f2(b[n]), acc[i][n]);
        }
    }
    // Every group's sums into its block's shared memory, [pair of rows][column][thread]; then
    // each block of the cluster finishes its part of the row pairs.
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    uint64_t *sum = reinterpret_cast<uint64_t *>(dyn);
    constexpr int PART = 32 * GROUP;  // of a group
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 8; ++n) sum[group * PART + (i * 8 + n) * GROUP + t] = acc[i][n].v;
    cluster_sync();
    // 4 columns (of g and of u) of a row pair a thread, over all threads of the cluster
    constexpr int HALVES = GATED ? 1 : 2;
    for (int e = rank * THREADS + (int)threadIdx.x; e < 4 * HALVES * GROUP; e += THREADS * share) {
        const int t2 = e % GROUP, i = e / GROUP % 4, half = e / GROUP / 4;
        F2 v[GATED ? 8 : 4];
#pragma unroll
        for (int n = 0; n < (GATED ? 8 : 4); ++n) {
            const uint64_t *at = sum + (i * 8 + half * 4 + n) * GROUP + t2;
            v[n] = f2(0.0f);
            for (int r = 0; r < share; ++r)
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    F2 x;
                    x.v = load_of_rank(at + g * PART, r);
                    v[n] = add2(v[n], x);
                }
        }
        const int m = m0 + t2 / 8 * 4 + (i & 1) * 2 + (i >> 1) * 64;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + half * 32 + t2 % 8 * 4 + j;
            if (n >= p.N) break;
            float d[2], du[2];
            split(v[j], d[0], d[1]);
            if (GATED) split(v[GATED ? 4 + j : j], du[0], du[1]);
#pragma unroll
            for (int row = 0; row < 2; ++row) {
                if (m + row >= p.M) break;
                float *out = static_cast<float *>(z ? p.out2 : p.out) + (int64_t)(m + row) * p.ldo + n;
                float *a_at = static_cast<float *>(p.kept) +  (int64_t)(m + row) * p.N + n, *b_at = a_at + (int64_t)p.M * p.N;
                if (EPI == EPI_STORE) {
                    *out = d[row];
                } else if (GATED) {
                    float a = act_value<ACT>(d[row]), s;
                    *out = a * du[row];
                    if (p.kept) {
                        act_both<ACT>(d[row], a, s);
                        *a_at = a, *b_at = du[row] * s;
                    }
                } else {
                    *out = d[row] * *b_at;
                    static_cast<float *>(p.out2)[(int64_t)(m + row) * p.ldo + n] = d[row] * *a_at;
                }
            }
        }
    }
    cluster_sync();  // the others' shared memory is read no more
}

template <bool AK, bool BKM, int EPI, int ACT>
cudaError_t launch(const Product &p, cudaStream_t st) {
    constexpr int COLS = EPI == EPI_GATED ? BN / 2 : BN;
    const int64_t tm = (p.M + BM - 1) / BM, tn = (p.N + COLS - 1) / COLS, blocks = tm * tn * (p.batch ? 2 : 1);
    if (blocks > 0x7fffffff / 8) return cudaErrorInvalidValue;
    auto kernel = simt_product<AK, BKM, EPI, ACT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    // Blocks of a tile: an SM's blocks share its FMA rate, so a launch takes as long as the
    // fullest SM's blocks one after the other, each with its K blocks and about 8 more for its
    // start and end.
    const int64_t kb = (int64_t)((p.K + BK - 1) / BK) * (EPI != EPI_GATED && !p.batch && p.a1.p ? 2 : 1);
    int share = 1;
    int64_t best = 0;
    for (int s = 1; s <= 8; ++s) {
        const int64_t cost = (blocks * s + 151) / 152 * (kb / s + 8);
        if (best == 0 || cost < best) best = cost, share = s;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * share));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)share;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, (int)tn, (int)(tm * tn), share);
}

}  // namespace

cudaError_t launch_simt(const Product &p, cudaStream_t st) {
    cudaError_t e = cudaErrorInvalidValue;
    if (p.epi == EPI_GATED)
        with_act(p.act, [&](auto a) { e = launch<true, true, EPI_GATED, decltype(a)::value>(p, st); });
    else if (p.epi == EPI_DGATED)
        e = launch<true, false, EPI_DGATED, 0>(p, st);
    else if (p.a0.k_major)
        e = p.b0.k_major ? launch<true, true, EPI_STORE, 0>(p, st) : launch<true, false, EPI_STORE, 0>(p, st);
    else
        e = launch<false, false, EPI_STORE, 0>(p, st);
    return e;
}

}  // namespace ffn
}  // namespace im2win
