// Group norm: argument checks and buffers.
#include <initializer_list>

#include "group_norm.cuh"

using namespace im2win;
using namespace im2win::gnorm;

namespace {

im2win_status check_dims(int64_t N, int64_t P, int64_t C, int64_t G, int dtype) {
    if (N < 0 || P < 0 || C < 1 || G < 1 || elem_size(dtype) == 0 || C % G != 0) return IM2WIN_ERR_INVALID_ARG;
    const int64_t most = int64_t(1) << 31;
    if (N >= most || P >= most || C > (int64_t(1) << 20) || N * P > (int64_t(1) << 40) / C || N * C > (int64_t(1) << 31))
        return IM2WIN_ERR_UNSUPPORTED;
    return IM2WIN_OK;
}

bool known_act(int act) {
    return act == IM2WIN_ACT_NONE || with_act(act, [](auto) {});
}

// maps: tensors that a pass keeps on the chip, if it can (forward 1, backward 2).
GroupArgs make(int64_t N, int64_t P, int64_t C, int64_t G, int act, int dtype, int maps) {
    GroupArgs a = {};
    a.N = N, a.P = P, a.C = (int)C, a.G = (int)G, a.D = (int)(C / G), a.act = act;
    if (cut_rows(a, elem_size(dtype))) return a;
    if (!cut_resident(a, elem_size(dtype), maps)) cut(a, elem_size(dtype), maps);
    a.part_rows = N * a.chunks;
    a.folds = folds_of(a.part_rows);
    return a;
}

// The workspace: partial sums, and the groups' sums (backward) or their statistics (forward, where the
// caller keeps none); backward, runs of the partial sums. A forward call that reads its maps once needs none.
struct Parts {
    size_t part, sums, folded, bytes;
    Parts(const GroupArgs &a, bool backward) {
        part = 0;
        const bool once = a.resident || a.lanes;  // read once, in one launch
        sums = once && !backward ? 0 : round_up((size_t)(2 * a.part_rows) * a.C * 4, 256);
        folded = sums + (once ? 0 : round_up((size_t)(a.N * a.G) * 8, 256));
        bytes = folded + (backward ? round_up((size_t)2 * a.folds * a.C * 4, 256) : 0);
    }
};

void place(GroupArgs &a, const Parts &parts, void *ws, void *stats) {
    unsigned char *base = static_cast<unsigned char *>(ws);
    a.part = reinterpret_cast<float *>(base + parts.part);
    a.sums = reinterpret_cast<float *>(base + parts.sums);
    a.folded = reinterpret_cast<float *>(base + parts.folded);
    a.stats = static_cast<float *>(stats || a.resident || a.lanes ? stats : base + parts.sums);
}

}  // namespace

extern "C" {

im2win_status im2win_group_norm_size(int backward, int64_t N, int64_t P, int64_t C, int64_t G, int dtype, size_t *bytes) {
    if (!bytes) return IM2WIN_ERR_INVALID_ARG;
    const im2win_status s = check_dims(N, P, C, G, dtype);
    if (s == IM2WIN_OK) *bytes = N * P == 0 ? 0 : Parts(make(N, P, C, G, 0, dtype, backward ? 2 : 1), backward != 0).bytes;
    return s;
}

im2win_status im2win_group_norm(const void *x, const void *w, const void *b, void *y, void *stats, void *ws,
                                size_t ws_bytes, int64_t N, int64_t P, int64_t C, int64_t G, int act, double eps,
                                int dtype, void *stream) {
    const im2win_status s = check_dims(N, P, C, G, dtype);
    if (s != IM2WIN_OK) return s;
    if (!known_act(act) || !(eps >= 0.0)) return IM2WIN_ERR_INVALID_ARG;
    if (N * P == 0) return IM2WIN_OK;  // nothing to read or write
    if (!x || !y) return IM2WIN_ERR_INVALID_ARG;
    for (const void *p : {x, w, b, (const void *)y, (const void *)stats, (const void *)ws})
        if (!aligned_to(p, 16)) return IM2WIN_ERR_MISALIGNED;
    GroupArgs a = make(N, P, C, G, act, dtype, 1);
    const Parts parts(a, false);
    if (ws_bytes < parts.bytes || (!ws && parts.bytes)) return IM2WIN_ERR_WORKSPACE;
    a.x = x, a.w = w, a.b = b, a.y = y, a.eps = (float)eps;
    place(a, parts, ws, stats);
    cudaError_t e = cudaErrorInvalidValue;
    with_dtype(dtype, [&](auto *t) { e = launch_forward<std::remove_pointer_t<decltype(t)>>(a, static_cast<cudaStream_t>(stream)); });
    return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

im2win_status im2win_group_norm_backward(const void *dy, const void *x, const void *stats, const void *w, const void *b,
                                         void *dx, void *dw, void *db, void *ws, size_t ws_bytes, int64_t N, int64_t P,
                                         int64_t C, int64_t G, int act, int dtype, void *stream) {
    const im2win_status s = check_dims(N, P, C, G, dtype);
    if (s != IM2WIN_OK) return s;
    if (!known_act(act) || (dw && !w) || (db && !b)) return IM2WIN_ERR_INVALID_ARG;
    if (N * P > 0 && (!dy || !x || !stats)) return IM2WIN_ERR_INVALID_ARG;
    for (const void *p : {dy, x, w, b, (const void *)dx, (const void *)dw, (const void *)db, (const void *)ws})
        if (!aligned_to(p, 16)) return IM2WIN_ERR_MISALIGNED;
    if (!aligned_to(stats, 8)) return IM2WIN_ERR_MISALIGNED;  // (read in pairs: some images' part of a batch's)
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N * P == 0) {  // sums over nothing
        cudaError_t e = cudaSuccess;
        for (void *p : {dw, db})
            if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)C * elem_size(dtype), st);
        return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
    }
    if (!dx && !dw && !db) return IM2WIN_OK;
    GroupArgs a = make(N, P, C, G, act, dtype, 2);
    const Parts parts(a, true);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    a.x = x, a.dy = dy, a.w = w, a.b = b, a.dx = dx, a.dw = dw, a.db = db;
    place(a, parts, ws, const_cast<void *>(stats));
    cudaError_t e = cudaErrorInvalidValue;
    with_dtype(dtype, [&](auto *t) { e = launch_backward<std::remove_pointer_t<decltype(t)>>(a, st); });
    return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

}  // extern "C"
