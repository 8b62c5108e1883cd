// What tests/test_block_plans.py asks the feed-forward's and the norms' host code about
// shapes; nothing here runs on a GPU.
#include "gated_ffn.cuh"
#include "residual_norm.cuh"

extern "C" {

// Columns of the one kernel's second product, or 0 where that kernel does not take the sizes.
int ffn_fused_columns(int64_t R, int C, int64_t F) {
    return im2win::ffn::fused_cost(R, C, F) > 0 ? im2win::ffn::fused_columns(C) : 0;
}

}  // extern "C"
