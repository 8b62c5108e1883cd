// Gated feed-forward grouped by expert: the pairs' plan, and the launchers of what moves rows
// to the experts and back.
#pragma once

#include "gated_ffn.cuh"

namespace im2win {
namespace ffn {

constexpr int MAX_CHOICES = 32;  // experts of a row

// T rows with k experts each make T k pairs. A pair whose expert is in [0, E) has a place among
// the grouped rows: the experts' rows one after another, each expert's in the order of its
// pairs and from a multiple of GROUP_ROWS on.
struct PairPlan {
    int32_t *begin;  // [E + 1], the last one the number of grouped rows with their padding
    int32_t *count;  // [E]
    int32_t *slot;   // [T k]: the pair's grouped row, or -1
    int32_t *pair;   // [rows]: the grouped row's pair, or -1 (padding)
};

// The most grouped rows that `pairs` pairs can make.
inline int64_t grouped_rows(int64_t pairs, int64_t E) {
    return (pairs + (GROUP_ROWS - 1) * (pairs < E ? pairs : E) + GROUP_ROWS - 1) / GROUP_ROWS * GROUP_ROWS;
}
// Pairs a block of the planning kernels takes.
inline int64_t pairs_per_block(int64_t pairs) {
    const int64_t even = (pairs + 151) / 152;
    return even <= 2048 ? 2048 : (even + 255) / 256 * 256;
}

struct Rows {
    int64_t T, rows;  // rows of the call, and a bound of the grouped ones
    int k, E, C;
    int64_t Cp;       // pitch of grouped rows
    PairPlan plan;
};

// The plan; clears the status. hist: an int for each expert and block, where there are several blocks.
cudaError_t launch_plan(const Rows &r, const int32_t *experts, int32_t *hist, uint32_t *status, cudaStream_t st);
// grouped[row] = x[pair / k], zero in the padding; fp32: in three bf16 planes. scale[row] (where not
// null) = weights[pair].
cudaError_t launch_gather(const Rows &r, const void *x, const void *weights, void *grouped, float *scale, int dtype,
                          cudaStream_t st);
// The same of dy; dweights[pair] (where not null) = dy[pair / k] . ys[row], or zero without a row.
// Clears the status.
cudaError_t launch_gather_back(const Rows &r, const void *dy, const void *weights, const float *ys, void *grouped,
                               float *scale, void *dweights, uint32_t *status, int dtype, cudaStream_t st);
// out[t] = sum over the row's choices of weights (null: 1) * ys[slot], in their order.
cudaError_t launch_combine(const Rows &r, const float *ys, const void *weights, void *out, int dtype, cudaStream_t st);

// Inference of few rows: up to FEW_PAIRS pairs. h and its remainder h_lo (16-bit types) have T k rows of
// ldh elements, a multiple of 8 there.
constexpr int FEW_PAIRS = 64;
struct ExpertFew {
    int T, k, E, C, F, act;
    const void *x, *weights, *w_gate, *w_up, *w_down;
    const int32_t *experts;
    void *y, *h, *h_lo;
    int64_t ldh;
    uint32_t *status;
};
cudaError_t launch_expert_few(const ExpertFew &f, int dtype, cudaStream_t st);

}  // namespace ffn
}  // namespace im2win
