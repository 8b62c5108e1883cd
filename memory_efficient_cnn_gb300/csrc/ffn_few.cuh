// What the feed-forward's kernels of few rows share: a block's warps split the summed index of a few
// weight rows, whose bytes they copy ahead.
#pragma once

#include "gated_ffn.cuh"
#include "tc_ptx.cuh"

namespace im2win {
namespace ffn {
namespace {

constexpr int WARPS = 8, THREADS = 32 * WARPS;

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

}  // namespace
}  // namespace ffn
}  // namespace im2win
