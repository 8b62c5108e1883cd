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
    EPI_GATED = 1,  // two accumulators g, u: out[m][n] = act(g) * u; act(g) and u act'(g) kept where asked
    EPI_DGATED = 2  // d = dh: out = dg = d * u act'(g), out2 = du = d * act(g), from the kept values
};

// What a training step keeps of an M x N product: a = act(g) and b = u act'(g).
//
// 16-bit types: in 24 bits, the upper ones of their fp32 form. dg and du, made of
// them, are rounded to 8 or 11 bits on their own, and the 16 kept bits add less
// than a hundredth to that; 16-bit a and b would have added half. They lie in
// blocks of 32 rows by 8 columns: 16 bytes a row of a's upper halves, the same of
// b's, then 16 bytes a row of the next bytes, a's and b's, so that a warp whose
// lanes hold a row each moves 512 contiguous bytes.
//
// fp32: in fp32, row by row, all a before all b.
constexpr int KEPT_BLOCK = 1536;
__host__ __device__ inline int64_t kept_block(int m, int n, int N) {
    return ((int64_t)(m / 32) * ((N + 7) / 8) + n / 8) * KEPT_BLOCK + (m % 32) * 16;
}
inline size_t kept_bytes(int64_t M, int64_t N, bool f32) {
    return f32 ? (size_t)(M * N) * 8 : (size_t)((M + 31) / 32) * (size_t)((N + 7) / 8) * KEPT_BLOCK;
}

// D[M][N] = A0 B0^T (+ A1 B1^T); EPI_GATED: g = A0 B0^T, u = A0 B1^T; batch: out =
// A0 B0^T and out2 = A1 B1^T.
struct Product {
    int M = 0, N = 0, K = 0;
    Operand a0, b0, a1, b1;
    int epi = EPI_STORE;
    int act = 0;
    bool batch = false;
    void *out = nullptr, *out2 = nullptr;
    void *kept = nullptr;  // written (EPI_GATED, may be null) or read (EPI_DGATED)
    int64_t ldo = 0;       // row pitch of out and out2 in elements
};

// CUDA cores, fp32.
cudaError_t launch_simt(const Product &p, cudaStream_t st);

// Tensor cores: fp16/bf16; operands 16-byte aligned with pitches that are multiples
// of 8 elements. A product takes part_bytes of scratch. status: the workspace's
// status block, cleared first where asked.
struct TcPlan {
    int cg = 0, bn = 0;       // CTAs and columns of a tile
    bool streamed = false;    // K blocks dealt out evenly, partial tiles joined
    int tiles_m = 0, tiles_n = 0, units = 0, slots = 0;
    int64_t part_ld = 0, part_step = 0;
    size_t part_bytes = 0;
};
TcPlan plan_tc(const Product &p);
cudaError_t launch_tc(const Product &p, bool bf16, uint32_t *status, bool clear_status, void *part, cudaStream_t st);

// The forward pass of few rows (where is_few), from dense matrices of any
// alignment that their type allows; h and its remainder h_lo (16-bit types) have
// rows of ldh elements, a multiple of 8 there.
struct Few {
    int R, C, F, act;
    const void *x, *w_gate, *w_up, *w_down;
    void *y, *h, *h_lo;
    int64_t ldh;
    void *kept;
    uint32_t *status;
};
bool is_few(int64_t R, int64_t C, int64_t F, int dtype);
cudaError_t launch_few(const Few &f, int dtype, cudaStream_t st);

// Copies of dense matrices to a pitch that is a multiple of 8 elements (16-bit types).
struct Repitch {
    const void *src;
    void *dst;
    int rows, cols;
};
cudaError_t launch_repitch(const Repitch *list, int count, cudaStream_t st);  // count <= 5

}  // namespace ffn
}  // namespace im2win
