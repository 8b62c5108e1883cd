// The norms around a residual block with its gate and residual scale:
//   r = res_scale * x + gate * post(y),  n = pre(r),  and the gradients.
//
// With m, i the mean (0 for RMS) and inverse deviation of a row v, its normed
// row is hat = (v - m) i and post(v) = hat * w + b; for a gradient d of post(v),
//   e = d * w,  dv = i (e - [mean(e)] - hat * mean(e * hat)),
// the bracket for LAYER only. dt = dr + pre'(dn) is the gradient of r.
#include <algorithm>
#include <initializer_list>

#include "elem.cuh"

using namespace im2win;

namespace {

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

constexpr int ROW_THREADS = 256;

// Sum over the block, the same for every thread and in a fixed order.
__device__ __forceinline__ float block_sum(float v, float *s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < ROW_THREADS / 32; ++i) t += s[i];
    __syncthreads();
    return t;
}

template <typename T>
__device__ __forceinline__ float load_or(const void *p, int64_t i, float absent) {
    return p ? to_f32(static_cast<const T *>(p)[i]) : absent;
}

// Mean and inverse deviation of f(c), c < C, for a norm kind.
template <typename Fn>
__device__ __forceinline__ void row_moments(int kind, int64_t C, float eps, float *s, Fn f, float &m, float &i) {
    m = 0.0f, i = 1.0f;
    if (kind == IM2WIN_NORM_NONE) return;
    float a = 0.0f;
    if (kind == IM2WIN_NORM_LAYER) {
        for (int64_t c = threadIdx.x; c < C; c += ROW_THREADS) a += f(c);
        m = block_sum(a, s) / (float)C;
        a = 0.0f;
    }
    for (int64_t c = threadIdx.x; c < C; c += ROW_THREADS) {
        const float d = f(c) - m;
        a = fmaf(d, d, a);
    }
    i = 1.0f / sqrtf(block_sum(a, s) / (float)C + eps);
}

// One row of r in fp32, element by element.
template <typename T>
struct RowOf {
    const NormArgs &p;
    int64_t row, gate_row;
    float my, iy;
    __device__ RowOf(const NormArgs &p_, int64_t row_) : p(p_), row(row_), gate_row(row_ / p_.per_gate), my(0), iy(1) {}
    __device__ float x(int64_t c) const { return to_f32(static_cast<const T *>(p.x)[row * p.C + c]); }
    __device__ float y(int64_t c) const { return to_f32(static_cast<const T *>(p.y)[row * p.C + c]); }
    __device__ float yhat(int64_t c) const { return (y(c) - my) * iy; }
    __device__ float post(int64_t c) const {
        return fmaf(yhat(c), load_or<T>(p.w_post, c, 1.0f), load_or<T>(p.b_post, c, 0.0f));
    }
    __device__ float gate(int64_t c) const { return load_or<T>(p.gate, gate_row * p.C + c, 1.0f); }
    __device__ float r(int64_t c) const {
        const float kept = x(c) * load_or<T>(p.res_scale, c, 1.0f);
        return p.y ? fmaf(gate(c), post(c), kept) : kept;
    }
};

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) norm_forward(NormArgs p) {
    __shared__ float s[ROW_THREADS / 32];
    RowOf<T> row(p, blockIdx.x);
    if (p.y) row_moments(p.post, p.C, p.eps, s, [&](int64_t c) { return row.y(c); }, row.my, row.iy);
    float mr, ir;
    row_moments(p.pre, p.C, p.eps, s, [&](int64_t c) { return row.r(c); }, mr, ir);
    for (int64_t c = threadIdx.x; c < p.C; c += ROW_THREADS) {
        const float r = row.r(c);
        if (p.r) static_cast<T *>(p.r)[row.row * p.C + c] = from_f32<T>(r);
        if (p.n)
            static_cast<T *>(p.n)[row.row * p.C + c] =
                from_f32<T>(fmaf((r - mr) * ir, load_or<T>(p.w_pre, c, 1.0f), load_or<T>(p.b_pre, c, 0.0f)));
    }
}

// dt of one element of a row whose statistics are known.
template <typename T>
__device__ __forceinline__ float total_grad(const NormArgs &p, const RowOf<T> &row, const RowStats &st, int64_t c) {
    float dt = load_or<T>(p.dr, p.dr ? row.row * p.C + c : 0, 0.0f);
    if (p.dn) {
        const float e = to_f32(static_cast<const T *>(p.dn)[row.row * p.C + c]) * load_or<T>(p.w_pre, c, 1.0f);
        dt += st.ir * (e - st.e1 - (row.r(c) - st.mr) * st.ir * st.e2);
    }
    return dt;
}

template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) norm_backward_rows(NormArgs p) {
    __shared__ float s[ROW_THREADS / 32];
    RowOf<T> row(p, blockIdx.x);
    RowStats st = {};
    if (p.y) row_moments(p.post, p.C, p.eps, s, [&](int64_t c) { return row.y(c); }, row.my, row.iy);
    st.my = row.my, st.iy = row.iy;
    if (p.dn) {
        row_moments(p.pre, p.C, p.eps, s, [&](int64_t c) { return row.r(c); }, st.mr, st.ir);
        float a = 0.0f, b = 0.0f;
        for (int64_t c = threadIdx.x; c < p.C; c += ROW_THREADS) {
            const float e = to_f32(static_cast<const T *>(p.dn)[row.row * p.C + c]) * load_or<T>(p.w_pre, c, 1.0f);
            a += e;
            b = fmaf(e, (row.r(c) - st.mr) * st.ir, b);
        }
        if (p.pre == IM2WIN_NORM_LAYER) st.e1 = block_sum(a, s) / (float)p.C;
        st.e2 = block_sum(b, s) / (float)p.C;
    }
    if (threadIdx.x == 0) reinterpret_cast<RowStats *>(p.stats)[row.row] = st;
    float e1 = 0.0f, e2 = 0.0f;  // of post
    if (p.dy && p.post != IM2WIN_NORM_NONE) {
        float a = 0.0f, b = 0.0f;
        for (int64_t c = threadIdx.x; c < p.C; c += ROW_THREADS) {
            const float e = total_grad(p, row, st, c) * row.gate(c) * load_or<T>(p.w_post, c, 1.0f);
            a += e;
            b = fmaf(e, row.yhat(c), b);
        }
        if (p.post == IM2WIN_NORM_LAYER) e1 = block_sum(a, s) / (float)p.C;
        e2 = block_sum(b, s) / (float)p.C;
    }
    for (int64_t c = threadIdx.x; c < p.C; c += ROW_THREADS) {
        const float dt = total_grad(p, row, st, c);
        if (p.dx) static_cast<T *>(p.dx)[row.row * p.C + c] = from_f32<T>(dt * load_or<T>(p.res_scale, c, 1.0f));
        if (p.dy) {
            const float e = dt * row.gate(c);
            static_cast<T *>(p.dy)[row.row * p.C + c] = from_f32<T>(
                p.post == IM2WIN_NORM_NONE
                    ? e
                    : st.iy * (e * load_or<T>(p.w_post, c, 1.0f) - e1 - row.yhat(c) * e2));
        }
    }
}

// ---- sums over rows
enum Sum { SUM_RES, SUM_W_POST, SUM_B_POST, SUM_W_PRE, SUM_B_PRE, SUM_GATE, SUMS };

// The rows are cut into tasks, each within one gate group (group_splits > 1
// tasks of `span` rows a group) or of whole groups (group_splits = 1), so that
// a group's sum is either joined from its tasks' or written by its task.
struct SumPlan {
    int64_t groups, span, group_splits, groups_per_task, tasks;
};

SumPlan plan_sums(int64_t R, int64_t per_gate) {
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

constexpr int SUM_COLS = 32, SUM_LANES = 8;

// Block (column block, task): 32 columns, 8 rows at a time.
template <typename T>
__global__ void __launch_bounds__(SUM_COLS * SUM_LANES)
    norm_column_sums(NormArgs p, SumPlan plan, int64_t col_blocks, float *part, T *dgate) {
    __shared__ float s[SUMS][SUM_LANES][SUM_COLS];
    const int64_t task = blockIdx.x / col_blocks, c = (int64_t)(blockIdx.x % col_blocks) * SUM_COLS + threadIdx.x % SUM_COLS;
    const int lane = threadIdx.x / SUM_COLS;
    const bool in = c < p.C;
    float acc[SUMS] = {};
    auto join = [&](int q) {  // the column's sum over the lanes, in the first lane
        s[q][lane][threadIdx.x % SUM_COLS] = acc[q];
        acc[q] = 0.0f;
        __syncthreads();
        float t = 0.0f;
        if (lane == 0)
            for (int l = 0; l < SUM_LANES; ++l) t += s[q][l][threadIdx.x];
        __syncthreads();
        return t;
    };
    const int64_t g0 = plan.group_splits > 1 ? task / plan.group_splits : task * plan.groups_per_task;
    const int64_t g1 = min(plan.groups, g0 + plan.groups_per_task);
    for (int64_t g = g0; g < g1; ++g) {
        const int64_t first = g * p.per_gate + (plan.group_splits > 1 ? (task % plan.group_splits) * plan.span : 0);
        const int64_t last = min(min(p.R, (g + 1) * p.per_gate), plan.group_splits > 1 ? first + plan.span : p.R);
        for (int64_t r = first + lane; in && r < last; r += SUM_LANES) {
            RowOf<T> row(p, r);
            const RowStats st = reinterpret_cast<const RowStats *>(p.stats)[r];
            row.my = st.my, row.iy = st.iy;
            const float dt = total_grad(p, row, st, c);
            acc[SUM_RES] = fmaf(row.x(c), dt, acc[SUM_RES]);
            if (p.y) {
                acc[SUM_GATE] = fmaf(row.post(c), dt, acc[SUM_GATE]);
                const float dp = dt * row.gate(c);
                acc[SUM_W_POST] = fmaf(dp, row.yhat(c), acc[SUM_W_POST]);
                acc[SUM_B_POST] += dp;
            }
            if (p.dn) {
                const float d = to_f32(static_cast<const T *>(p.dn)[r * p.C + c]);
                acc[SUM_W_PRE] = fmaf(d, (row.r(c) - st.mr) * st.ir, acc[SUM_W_PRE]);
                acc[SUM_B_PRE] += d;
            }
        }
        if (dgate && plan.group_splits == 1) {
            const float t = join(SUM_GATE);
            if (lane == 0 && in) dgate[g * p.C + c] = from_f32<T>(t);
        }
    }
    for (int q = 0; q < SUMS; ++q) {
        const float t = join(q);
        if (lane == 0 && in) part[(q * plan.tasks + task) * p.C + c] = t;
    }
}

// out[j][c] = sum of the `per` partial rows of j, in their order.
template <typename T>
__global__ void __launch_bounds__(256) join_partials(const float *part, int64_t per, int64_t total, int64_t C, T *out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const float *src = part + (i / C) * per * C + i % C;
    float t = 0.0f;
    for (int64_t k = 0; k < per; ++k) t += src[k * C];
    out[i] = from_f32<T>(t);
}

im2win_status check_common(const NormArgs &p, int dtype, bool with_data) {
    if (p.R < 0 || p.C < 1 || p.per_gate < 1 || elem_size(dtype) == 0) return IM2WIN_ERR_INVALID_ARG;
    if (p.R > 0x7fffffff || p.C > (1 << 20) || p.R * p.C > (int64_t(1) << 40)) return IM2WIN_ERR_UNSUPPORTED;
    if (!with_data) return IM2WIN_OK;
    for (const int kind : {p.post, p.pre})
        if (kind < IM2WIN_NORM_NONE || kind > IM2WIN_NORM_LAYER) return IM2WIN_ERR_INVALID_ARG;
    if (!(p.eps >= 0.0f)) return IM2WIN_ERR_INVALID_ARG;
    if (p.post == IM2WIN_NORM_NONE && p.w_post) return IM2WIN_ERR_INVALID_ARG;
    if (p.pre == IM2WIN_NORM_NONE && p.w_pre) return IM2WIN_ERR_INVALID_ARG;
    if ((p.post != IM2WIN_NORM_LAYER && p.b_post) || (p.pre != IM2WIN_NORM_LAYER && p.b_pre))
        return IM2WIN_ERR_INVALID_ARG;
    return IM2WIN_OK;
}

bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned_to(p, 16)) return false;
    return true;
}

struct BackwardParts {
    size_t stats, part, bytes;
    BackwardParts(int64_t R, int64_t C, const SumPlan &s) {
        stats = 0;
        part = round_up((size_t)R * sizeof(RowStats), 256);
        bytes = part + round_up((size_t)SUMS * s.tasks * C * 4, 256);
    }
};

}  // namespace

extern "C" {

im2win_status im2win_residual_norm(const void *x, const void *y, const void *gate, int64_t rows_per_gate,
                                   const void *res_scale, int post, const void *w_post, const void *b_post, int pre,
                                   const void *w_pre, const void *b_pre, double eps, void *r, void *n, int64_t R,
                                   int64_t C, int dtype, void *stream) {
    NormArgs p = {};
    p.x = x; p.y = y; p.gate = gate; p.res_scale = res_scale;
    p.w_post = w_post; p.b_post = b_post; p.w_pre = w_pre; p.b_pre = b_pre;
    p.post = post; p.pre = pre; p.eps = (float)eps;
    p.R = R; p.C = C; p.per_gate = rows_per_gate; p.r = r; p.n = n;
    const im2win_status s = check_common(p, dtype, true);
    if (s != IM2WIN_OK) return s;
    if (R == 0) return IM2WIN_OK;  // no rows: nothing to read or write
    if (!y && (post != IM2WIN_NORM_NONE || gate)) return IM2WIN_ERR_INVALID_ARG;
    if (!x || (!r && !n) || (n != nullptr) != (pre != IM2WIN_NORM_NONE)) return IM2WIN_ERR_INVALID_ARG;
    if (!all_aligned({x, y, gate, res_scale, w_post, b_post, w_pre, b_pre, r, n})) return IM2WIN_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    with_dtype(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        norm_forward<T><<<(unsigned)R, ROW_THREADS, 0, st>>>(p);
    });
    return cudaGetLastError() == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

im2win_status im2win_residual_norm_backward_size(int64_t R, int64_t C, int64_t rows_per_gate, int dtype, size_t *bytes) {
    if (!bytes) return IM2WIN_ERR_INVALID_ARG;
    NormArgs p = {};
    p.R = R; p.C = C; p.per_gate = rows_per_gate;
    const im2win_status s = check_common(p, dtype, false);
    if (s != IM2WIN_OK) return s;
    *bytes = R == 0 ? 0 : BackwardParts(R, C, plan_sums(R, std::min(rows_per_gate, R))).bytes;
    return IM2WIN_OK;
}

im2win_status im2win_residual_norm_backward(const void *dr, const void *dn, const void *x, const void *y,
                                            const void *gate, int64_t rows_per_gate, const void *res_scale, int post,
                                            const void *w_post, const void *b_post, int pre, const void *w_pre,
                                            const void *b_pre, double eps, void *dx, void *dy, void *dgate,
                                            void *dres_scale, void *dw_post, void *db_post, void *dw_pre,
                                            void *db_pre, void *ws, size_t ws_bytes, int64_t R, int64_t C, int dtype,
                                            void *stream) {
    NormArgs p = {};
    p.x = x; p.y = y; p.gate = gate; p.res_scale = res_scale;
    p.w_post = w_post; p.b_post = b_post; p.w_pre = w_pre; p.b_pre = b_pre;
    p.post = post; p.pre = pre; p.eps = (float)eps;
    p.R = R; p.C = C; p.per_gate = rows_per_gate;
    p.dr = dr; p.dn = dn; p.dx = dx; p.dy = dy;
    const im2win_status s = check_common(p, dtype, true);
    if (s != IM2WIN_OK) return s;
    // a gradient of an absent input, and dn without its norm
    if ((!res_scale && dres_scale) || (!w_post && dw_post) || (!b_post && db_post) || (!w_pre && dw_pre) ||
        (!b_pre && db_pre) || (pre == IM2WIN_NORM_NONE && dn))
        return IM2WIN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int esz = elem_size(dtype);
    if (!all_aligned({dr, dn, x, y, gate, res_scale, w_post, b_post, w_pre, b_pre, dx, dy, dgate, dres_scale, dw_post,
                      db_post, dw_pre, db_pre, ws}))
        return IM2WIN_ERR_MISALIGNED;
    if (R == 0) {  // sums over no rows
        cudaError_t e = cudaSuccess;
        for (void *w : {dres_scale, dw_post, db_post, dw_pre, db_pre})
            if (w && e == cudaSuccess) e = cudaMemsetAsync(w, 0, (size_t)C * esz, st);
        return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
    }
    if (!x || (!y && (post != IM2WIN_NORM_NONE || gate || dy)) || (!gate && dgate)) return IM2WIN_ERR_INVALID_ARG;
    p.per_gate = std::min(rows_per_gate, R);
    const SumPlan plan = plan_sums(R, p.per_gate);
    const BackwardParts parts(R, C, plan);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    const int64_t col_blocks = (C + SUM_COLS - 1) / SUM_COLS;
    if (plan.tasks * col_blocks > 0x7fffffff) return IM2WIN_ERR_UNSUPPORTED;
    p.stats = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + parts.stats);
    float *part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + parts.part);
    with_dtype(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        norm_backward_rows<T><<<(unsigned)R, ROW_THREADS, 0, st>>>(p);
        if (!dgate && !dres_scale && !dw_post && !db_post && !dw_pre && !db_pre) return;
        norm_column_sums<T><<<(unsigned)(plan.tasks * col_blocks), SUM_COLS * SUM_LANES, 0, st>>>(
            p, plan, col_blocks, part, static_cast<T *>(dgate));
        void *outs[SUMS] = {dres_scale, dw_post, db_post, dw_pre, db_pre, plan.group_splits > 1 ? dgate : nullptr};
        for (int q = 0; q < SUMS; ++q) {
            if (!outs[q]) continue;
            const int64_t total = q == SUM_GATE ? plan.groups * C : C;
            join_partials<T><<<(unsigned)((total + 255) / 256), 256, 0, st>>>(
                part + q * plan.tasks * C, q == SUM_GATE ? plan.group_splits : plan.tasks, total, C,
                static_cast<T *>(outs[q]));
        }
    });
    return cudaGetLastError() == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

}  // extern "C"
