// The norms around a residual block: argument checks and workspace sizes.
#include <initializer_list>

#include "residual_norm.cuh"

using namespace im2win;
using namespace im2win::rnorm;

namespace {

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
    cudaError_t e = cudaSuccess;
    with_dtype(dtype, [&](auto *t) { e = launch_norm_forward<std::remove_pointer_t<decltype(t)>>(p, st); });
    return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

im2win_status im2win_residual_norm_backward_size(int64_t R, int64_t C, int64_t rows_per_gate, int dtype, size_t *bytes) {
    if (!bytes) return IM2WIN_ERR_INVALID_ARG;
    NormArgs p = {};
    p.R = R; p.C = C; p.per_gate = rows_per_gate;
    const im2win_status s = check_common(p, dtype, false);
    if (s != IM2WIN_OK) return s;
    *bytes = R == 0 ? 0 : BackwardParts(R, C, std::min(rows_per_gate, R)).bytes;
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
    const BackwardParts parts(R, C, p.per_gate);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    const ColumnGrads g = {dgate, dres_scale, dw_post, db_post, dw_pre, db_pre};
    cudaError_t e = cudaSuccess;
    with_dtype(dtype, [&](auto *t) { e = launch_norm_backward<std::remove_pointer_t<decltype(t)>>(p, g, ws, st); });
    return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

}  // extern "C"
