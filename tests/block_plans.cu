// What tests/test_block_plans.py asks the feed-forward's and the norms' host code about
// shapes; nothing here runs on a GPU.
#include "gated_ffn.cuh"
#include "residual_norm.cuh"

extern "C" {

// Columns of the one kernel's second product, or 0 where that kernel does not take the sizes.
int ffn_fused_columns(int64_t R, int C, int64_t F) {
    return im2win::ffn::fused_cost(R, C, F) > 0 ? im2win::ffn::fused_columns(C) : 0;
}

// Blocks of the norms' backward pass in one reading (0: element by element); whether it takes whole groups.
int norm_back_blocks(int64_t R, int64_t C, int64_t per_gate, int *short_groups) {
    const im2win::rnorm::BackPlan b = im2win::rnorm::plan_back(R, C, per_gate);
    *short_groups = b.short_groups;
    return b.blocks;
}

}  // extern "C"
