// Gated feed-forward: the problem, its buffers and the launchers of its products.
#pragma once

#include "elem.cuh"

namespace im2win {
namespace ffn {

// R rows, C channels, F hidden channels. The products of a call, as
// D[M][N] = sum_k A(m, k) B(n, k):
//   forward   g, u = x w_gate^T, x w_up^T   (M = R, N = F, K = C), joined to h
//             y = h w_down^T                (M = R, N = C, K = F)
//   backward  dh = dy w_down                (M = R, N = F, K = C), made into dg, du
//             dx = dg w_gate + du w_up      (M = R, N = C, K = F, twice)
//             dw_gate = dg^T x, dw_up = du^T x   (M = F, N = C, K = R)
//             dw_down = dy^T h                   (M = C, N = F, K = R)
struct Dims {
    int R, C, F;
};

// One operand: element (i, k) (i an output row or column, k the summed index) is
// p[i * ld + k] (k_major) or p[k * ld + i].
struct Operand {
    const void *p = nullptr;
    int64_t ld = 0;
    bool k_major = true;
};

// What becomes of an accumulated element (m, n).
enum Epilogue {
    EPI_STORE = 0,  // out[m][n] = d
    EPI_GATED = 1,  // two accumulators g, u: out[m][n] = act(g) * u; g and u kept in fp32 where asked
    EPI_DGATED = 2  // d = dh: out = dg, out2 = du, from the kept g, u
};

// D[M][N] = A0 B0^T (+ A1 B1^T); EPI_GATED: g = A0 B0^T, u = A0 B1^T.
struct Product {
    int M = 0, N = 0, K = 0;
    Operand a0, b0, a1, b1;
    int epi = EPI_STORE;
    int act = 0;
    void *out = nullptr, *out2 = nullptr;
    float *g = nullptr, *u = nullptr;  // [M][N]: written (EPI_GATED, may be null) or read (EPI_DGATED)
    int64_t ldo = 0;                   // row pitch of out and out2 in elements
};

cudaError_t launch_simt(const Product &p, int dtype, cudaStream_t st);

}  // namespace ffn
}  // namespace im2win
