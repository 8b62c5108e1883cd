// Residual norm: the problem, how its sums over rows are cut, and the launchers
// (one translation unit for each type).
#pragma once

#include <algorithm>

#include "elem.cuh"

namespace im2win {
namespace rnorm {

struct NormArgs {
    const void *x, *y, *gate, *res_scale, *w_post, *b_post, *w_pre, *b_pre;
    int post, pre;
    float eps;
    int64_t R, C, per_gate;
    void *r, *n;                             // forward
    const void *dr, *dn;                     // backward
    void *dx, *dy;
    float *stats;                            // backward: per row, see RowStats
};

// What the backward pass's column sums need of a row.
struct RowStats {
    float my, iy, mr, ir, e1, e2;  // means and inverse deviations of y and r; mean(e) and mean(e * hat) of pre
};

enum Sum { SUM_RES, SUM_W_POST, SUM_B_POST, SUM_W_PRE, SUM_B_PRE, SUM_GATE, SUMS };

// The rows are cut into tasks, each within one gate group (group_splits > 1
// tasks of `span` rows a group) or of whole groups (group_splits = 1), so that
// a group's sum is either joined from its tasks' or written by its task.
struct SumPlan {
    int64_t groups, span, group_splits, groups_per_task, tasks;
};

inline SumPlan plan_sums(int64_t R, int64_t per_gate) {
    SumPlan s;
    const int64_t want = std::max<int64_t>(64, (R + 511) / 512);  // rows a task
    s.groups = (R + per_gate - 1) / per_gate;
    if (per_gate > want) {
        s.group_splits = (per_gate + want - 1) / want;
        s.span = (per_gate + s.group_splits - 1) / s.group_splits;
        s.groups_per_task = 1;
        s.tasks = s.groups * s.group_splits;
    } else {
        s.group_splits = 1;
        s.groups_per_task = want / per_gate;
        s.span = s.groups_per_task * per_gate;
        s.tasks = (s.groups + s.groups_per_task - 1) / s.groups_per_task;
    }
    return s;
}

// The fused backward pass, which reads its inputs once, and its cut:
//  long groups   block k takes rows [R k / blocks, R (k+1) / blocks);
//  short groups  a row slot takes whole gate groups.
struct BackPlan {
    int tpr = 0, ept = 0, threads = 0, blocks = 0;
    bool short_groups = false;
    int64_t groups = 0, segments = 0;  // segments: long groups' A and B
};
enum BackSum { BACK_RES, BACK_W_PRE, BACK_B_PRE, BACK_A, BACK_B, BACK_SUMS };

constexpr int SMS = 152;  // blocks are cut for this many SMs, so that results depend on the shape alone
constexpr int FUSED_THREADS = 512;

// The fused pass holds rows of up to 4096 elements (8 a thread), or 8192 (16 a thread).
inline BackPlan plan_back(int64_t R, int64_t C, int64_t per_gate) {
    BackPlan b;
    if (R == 0 || C > 16 * FUSED_THREADS) return b;
    b.ept = C > 8 * FUSED_THREADS ? 16 : 8;
    b.threads = FUSED_THREADS;
    b.tpr = 8;
    while (b.tpr * b.ept < C) b.tpr *= 2;
    const int64_t rpb = b.threads / b.tpr;
    b.groups = (R + per_gate - 1) / per_gate;
    b.blocks = (int)std::min<int64_t>(SMS, (R + rpb - 1) / rpb);
    // Rounds of a slot: long groups end with two joins, about a round's time each. Both forms read rows
    // once; 4096 x 8192 bf16, RMS: 242 us with a gate a row in the short form and 2441 us in the long one,
    // a gate for 8 rows 192 us and 518 us; for 16 rows the rule takes the long one's 345 us, for 64 216 us.
    const int64_t slots = b.blocks * rpb;
    const int64_t long_rounds = (R + slots - 1) / slots + 2 * (b.groups / b.blocks + 1) + b.groups / b.blocks;
    const int64_t short_rounds = (b.groups + slots - 1) / slots * (per_gate + 1);
    b.short_groups = short_rounds < long_rounds;
    b.segments = b.short_groups ? 0 : b.groups + b.blocks;
    return b;
}

struct JoinOuts {
    void *out[BACK_SUMS];
    void *dgate;
};
// Scratch of the backward pass, in bytes from its start.
struct BackwardParts {
    size_t stats, part, seg, bytes;
    BackwardParts(int64_t R, int64_t C, int64_t per_gate) {
        const BackPlan f = plan_back(R, C, per_gate);
        stats = 0;
        part = f.blocks ? 0 : round_up((size_t)R * sizeof(RowStats), 256);
        const int64_t rows = f.blocks ? (int64_t)BACK_SUMS * f.blocks : (int64_t)SUMS * plan_sums(R, per_gate).tasks;
        seg = part + round_up((size_t)rows * C * 4, 256);
        bytes = seg + round_up((size_t)f.segments * 2 * C * 4, 256);
    }
};

template <typename T>
cudaError_t launch_norm_forward(const NormArgs &p, cudaStream_t st);

// Gradients of p.R >= 1 rows; any of the outputs may be null.
struct ColumnGrads {
    void *dgate, *dres_scale, *dw_post, *db_post, *dw_pre, *db_pre;
    bool any() const { return dgate || dres_scale || dw_post || db_post || dw_pre || db_pre; }
};
template <typename T>
cudaError_t launch_norm_backward(const NormArgs &p, const ColumnGrads &g, void *ws, cudaStream_t st);

}  // namespace rnorm
}  // namespace im2win
