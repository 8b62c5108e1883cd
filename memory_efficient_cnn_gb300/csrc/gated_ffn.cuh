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

// One operand: element (i, k) (i an output row or column, k the summed index) is
// p[i * ld + k] (k_major) or p[k * ld + i].
struct Operand {
    const void *p = nullptr;
    int64_t ld = 0;
    bool k_major = true;
    int64_t plane = 0;  // fp32 in three bf16 planes: elements from one to the next
};

// 16-bit types round h, dg and du to the type: they are operands of 16-bit products, and a
// remainder beside them would double those products' work and the bytes of h. y is then
// 2.3e-3 (bf16) or 2.9e-4 (fp16) off in the 2-norm where h in fp32 gives 1.7e-3 or 2.1e-4, the
// output's own rounding. Few rows, bound by the weights, keep the remainder of h.

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
// fp32: in fp32, blocks of 32 rows by 4 columns, 16 bytes a row, all a before all b.
constexpr int KEPT_BLOCK = 1536;
__host__ __device__ inline int64_t kept_block(int m, int n, int N) {
    return ((int64_t)(m / 32) * ((N + 7) / 8) + n / 8) * KEPT_BLOCK + (m % 32) * 16;
}
__host__ __device__ inline int64_t kept_index_f32(int m, int n, int N) {
    return ((int64_t)(m / 32) * ((N + 3) / 4) + n / 4) * 128 + (m % 32) * 4 + n % 4;
}
__host__ __device__ inline int64_t kept_count_f32(int64_t M, int64_t N) { return (M + 31) / 32 * ((N + 3) / 4) * 128; }
inline size_t kept_bytes(int64_t M, int64_t N, bool f32) {
    return f32 ? (size_t)kept_count_f32(M, N) * 8 : (size_t)((M + 31) / 32) * (size_t)((N + 7) / 8) * KEPT_BLOCK;
}

// An fp32 value as three bf16 ones: the upper 16 bits (cut, so that they cannot
// round to infinity), the rest rounded, and what is left rounded: v = h + m + l to
// 2^-26 of v. Infinities and NaN stand in h alone.
__device__ __forceinline__ void split_f32(float v, uint16_t &h, uint16_t &m, uint16_t &l) {
    const uint32_t bits = __float_as_uint(v);
    if ((bits & 0x7f800000u) == 0x7f800000u) {
        h = __bfloat16_as_ushort(__float2bfloat16_rn(v)), m = l = 0;
        return;
    }
    const float rest = v - __uint_as_float(bits & 0xffff0000u);
    const bf16_t mid = __float2bfloat16_rn(rest);
    h = (uint16_t)(bits >> 16);
    m = __bfloat16_as_ushort(mid);
    l = __bfloat16_as_ushort(__float2bfloat16_rn(rest - __bfloat162float(mid)));
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
    int64_t plane = 0;     // fp32, GATED and DGATED: elements from one plane of out and out2 to the next
};

// Tensor cores: fp16/bf16; operands 16-byte aligned with pitches that are multiples
// of 8 elements. A product takes part_bytes of scratch. status: the workspace's
// status block; first: the call's first product, which clears it.
struct TcPlan {
    int cg = 0, bn = 0;       // CTAs and columns of a tile
    bool streamed = false;    // K blocks dealt out evenly, partial tiles joined
    int tiles_m = 0, tiles_n = 0, units = 0, slots = 0;
    int64_t part_ld = 0, part_step = 0;
    size_t part_bytes = 0;
    double cost = 0;          // estimated microseconds
};
TcPlan plan_tc(const Product &p);
cudaError_t launch_tc(const Product &p, bool bf16, uint32_t *status, bool first, void *part, cudaStream_t st);

// The same for fp32, whose operands are three bf16 planes each (h + m + l, see
// split_f32): GATED and DGATED write such planes, STORE writes fp32.
TcPlan plan_f32(const Product &p);
cudaError_t launch_f32(const Product &p, uint32_t *status, bool first, void *part, cudaStream_t st);

// The forward pass of few rows (where is_few), from dense matrices of any
// alignment that their type allows; h and its remainder h_lo (16-bit types) have
// rows of ldh elements, a multiple of 8 there.
struct Few {
    int R, C, F, act;
    const void *x, *w_gate, *w_up, *w_down;
    void *y, *h, *h_lo;
    int64_t ldh;
    uint16_t *planes;  // fp32, training: h in three planes of R rows of plane_ld elements
    int64_t plane_ld;
    void *kept;
    uint32_t *status;
};
bool is_few(int64_t R, int64_t C, int64_t F, int dtype);
cudaError_t launch_few(const Few &f, int dtype, cudaStream_t st);

// The forward pass of few channels (16-bit types) in one kernel, which keeps nothing:
// an estimate of its time, comparable with TcPlan's, or zero where it does not apply.
struct Fused {
    int R, C, F, act;
    Operand x, wg, wu, wd;  // pitches that are multiples of 8 elements
    void *y;
};
double fused_cost(int64_t R, int64_t C, int64_t F);
// Columns of its second product: a pair's 256-row product takes multiples of 32.
constexpr int fused_columns(int C) { return (C + 31) / 32 * 32; }
cudaError_t launch_fused(const Fused &f, bool bf16, uint32_t *status, cudaStream_t st);

// Copies of dense matrices to a pitch that is a multiple of 8 elements: 16-bit types
// as they are, fp32 in three bf16 planes.
struct Repitch {
    const void *src;
    void *dst;
    int rows, cols;
};
cudaError_t launch_repitch(const Repitch *list, int count, bool f32, cudaStream_t st);  // count <= 5

}  // namespace ffn
}  // namespace im2win
