// What tests/test_block_plans.py asks the feed-forward's and the norms' host code about
// shapes; nothing here runs on a GPU.
#include "gated_ffn.cuh"
#include "residual_norm.cuh"

extern "C" {

// Columns of the one kernel's second product, or 0 where that kernel does not take the sizes.
int ffn_fused_columns(int64_t R, int C, int64_t F) {
    return im2win::ffn::fused_cost(R, C, F) > 0 ? im2win::ffn::fused_columns(C) : 0;
}

// Tiles a unit (CTA or pair) at a time, and whether their K is dealt out; units 0: no plan. kind as in
// the epilogues; two: a second pair of operands, joined to the first (1) or apart (2).
int ffn_product_units(int f32, int M, int N, int K, int kind, int two, int *streamed) {
    im2win::ffn::Product p;
    const void *some = reinterpret_cast<const void *>(16);
    p.M = M, p.N = N, p.K = K, p.epi = kind, p.batch = two == 2;
    p.a0.p = p.b0.p = some;
    if (two || kind == im2win::ffn::EPI_GATED) p.b1.p = some;
    if (two) p.a1.p = some;
    const im2win::ffn::TcPlan pl = f32 ? im2win::ffn::plan_f32(p) : im2win::ffn::plan_tc(p);
    *streamed = pl.streamed;
    return pl.units;
}

// Blocks of the norms' backward pass in one reading (0: element by element); whether it takes whole groups.
int norm_back_blocks(int64_t R, int64_t C, int64_t per_gate, int *short_groups) {
    const im2win::rnorm::BackPlan b = im2win::rnorm::plan_back(R, C, per_gate);
    *short_groups = b.short_groups;
    return b.blocks;
}

}  // extern "C"
