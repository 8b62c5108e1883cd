// Gated feed-forward block: argument checks, buffers and the sequence of products.
#include "gated_ffn.cuh"

using namespace im2win;
using namespace im2win::ffn;

namespace {

im2win_status check_dims(int64_t R, int64_t C, int64_t F, int dtype) {
    if (R < 0 || C < 1 || F < 1 || elem_size(dtype) == 0) return IM2WIN_ERR_INVALID_ARG;
    const int64_t most = 0x7fffffff, area = int64_t(1) << 40;
    if (R > most || C > most || F > most || R * C > area || R * F > area || C * F > area) return IM2WIN_ERR_UNSUPPORTED;
    return IM2WIN_OK;
}

// Byte offsets of the parts of a buffer, each on a 256-byte boundary.
struct Parts {
    size_t end;
    explicit Parts(size_t begin) : end(begin) {}
    size_t add(size_t bytes) {
        const size_t at = end;
        end += round_up(bytes, 256);
        return at;
    }
};

// saved: h, then g and u in fp32.
struct SavedParts {
    size_t h, g, u, bytes;
    SavedParts(int64_t R, int64_t F, int esz) {
        Parts p(0);
        h = p.add((size_t)(R * F) * esz);
        g = p.add((size_t)(R * F) * 4);
        u = p.add((size_t)(R * F) * 4);
        bytes = p.end;
    }
};

struct ForwardParts {
    size_t h, bytes;
    ForwardParts(int64_t R, int64_t F, int esz, bool saved) {
        Parts p(kStatusBytes);
        h = p.end;
        if (!saved) p.add((size_t)(R * F) * esz);
        bytes = p.end;
    }
};

struct BackwardParts {
    size_t dg, du, bytes;
    BackwardParts(int64_t R, int64_t F, int esz) {
        Parts p(kStatusBytes);
        dg = p.add((size_t)(R * F) * esz);
        du = p.add((size_t)(R * F) * esz);
        bytes = p.end;
    }
};

unsigned char *at(void *base, size_t off) { return static_cast<unsigned char *>(base) + off; }
const unsigned char *at(const void *base, size_t off) { return static_cast<const unsigned char *>(base) + off; }

bool known_act(int act) {
    return with_act(act, [](auto) {});
}

}  // namespace

extern "C" {

im2win_status im2win_gated_ffn_size(int buffer, int64_t R, int64_t C, int64_t F, int dtype, size_t *bytes) {
    if (!bytes) return IM2WIN_ERR_INVALID_ARG;
    const im2win_status s = check_dims(R, C, F, dtype);
    if (s != IM2WIN_OK) return s;
    const int esz = elem_size(dtype);
    switch (buffer) {
        case IM2WIN_FFN_FORWARD: *bytes = ForwardParts(R, F, esz, false).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_TRAIN: *bytes = ForwardParts(R, F, esz, true).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_BACKWARD: *bytes = BackwardParts(R, F, esz).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_SAVED: *bytes = SavedParts(R, F, esz).bytes; return IM2WIN_OK;
        default: return IM2WIN_ERR_INVALID_ARG;
    }
}

im2win_status im2win_gated_ffn(const void *x, const void *w_gate, const void *w_up, const void *w_down, void *y,
                               void *saved, void *ws, size_t ws_bytes, int64_t R, int64_t C, int64_t F, int act,
                               int dtype, void *stream) {
    const im2win_status s = check_dims(R, C, F, dtype);
    if (s != IM2WIN_OK) return s;
    if (!known_act(act)) return IM2WIN_ERR_INVALID_ARG;
    if (R == 0) return IM2WIN_OK;  // no rows: nothing to read or write
    if (!x || !w_gate || !w_up || !w_down || !y) return IM2WIN_ERR_INVALID_ARG;
    for (const void *p : {x, w_gate, w_up, w_down, (const void *)y, (const void *)saved, (const void *)ws})
        if (!aligned_to(p, 16)) return IM2WIN_ERR_MISALIGNED;
    const int esz = elem_size(dtype);
    const ForwardParts parts(R, F, esz, saved != nullptr);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const SavedParts kept(R, F, esz);
    void *h = saved ? at(saved, kept.h) : at(ws, parts.h);

    cudaError_t e = cudaMemsetAsync(ws, 0, kStatusBytes, st);
    Product p1;
    p1.M = (int)R; p1.N = (int)F; p1.K = (int)C;
    p1.a0 = {x, C, true};
    p1.b0 = {w_gate, C, true};
    p1.b1 = {w_up, C, true};
    p1.epi = EPI_GATED; p1.act = act;
    p1.out = h; p1.ldo = F;
    if (saved) {
        p1.g = reinterpret_cast<float *>(at(saved, kept.g));
        p1.u = reinterpret_cast<float *>(at(saved, kept.u));
    }
    if (e == cudaSuccess) e = launch_simt(p1, dtype, st);
    Product p2;
    p2.M = (int)R; p2.N = (int)C; p2.K = (int)F;
    p2.a0 = {h, F, true};
    p2.b0 = {w_down, F, true};
    p2.out = y; p2.ldo = C;
    if (e == cudaSuccess) e = launch_simt(p2, dtype, st);
    return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

im2win_status im2win_gated_ffn_backward(const void *dy, const void *x, const void *w_gate, const void *w_up,
                                        const void *w_down, const void *saved, void *dx, void *dw_gate, void *dw_up,
                                        void *dw_down, void *ws, size_t ws_bytes, int64_t R, int64_t C, int64_t F,
                                        int act, int dtype, void *stream) {
    const im2win_status s = check_dims(R, C, F, dtype);
    if (s != IM2WIN_OK) return s;
    if (!known_act(act)) return IM2WIN_ERR_INVALID_ARG;
    const bool want_dw = dw_gate != nullptr;
    if ((dw_up != nullptr) != want_dw || (dw_down != nullptr) != want_dw) return IM2WIN_ERR_INVALID_ARG;
    if (R > 0 && (!dy || !x || !w_gate || !w_up || !w_down || !saved)) return IM2WIN_ERR_INVALID_ARG;
    for (const void *p : {dy, x, w_gate, w_up, w_down, saved, (const void *)dx, (const void *)dw_gate,
                          (const void *)dw_up, (const void *)dw_down, (const void *)ws})
        if (!aligned_to(p, 16)) return IM2WIN_ERR_MISALIGNED;
    const int esz = elem_size(dtype);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (R == 0) {  // sums over no rows
        for (void *w : {dw_gate, dw_up, dw_down})
            if (w && e == cudaSuccess) e = cudaMemsetAsync(w, 0, (size_t)(C * F) * esz, st);
        return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
    }
    if (!dx && !want_dw) return IM2WIN_OK;
    const BackwardParts parts(R, F, esz);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    const SavedParts kept(R, F, esz);
    void *dg = at(ws, parts.dg), *du = at(ws, parts.du);

    e = cudaMemsetAsync(ws, 0, kStatusBytes, st);
    Product p;
    p.M = (int)R; p.N = (int)F; p.K = (int)C;
    p.a0 = {dy, C, true};
    p.b0 = {w_down, F, false};
    p.epi = EPI_DGATED; p.act = act;
    p.out = dg; p.out2 = du; p.ldo = F;
    p.g = reinterpret_cast<float *>(const_cast<unsigned char *>(at(saved, kept.g)));
    p.u = reinterpret_cast<float *>(const_cast<unsigned char *>(at(saved, kept.u)));
    if (e == cudaSuccess) e = launch_simt(p, dtype, st);
    if (dx && e == cudaSuccess) {
        Product q;
        q.M = (int)R; q.N = (int)C; q.K = (int)F;
        q.a0 = {dg, F, true};
        q.b0 = {w_gate, C, false};
        q.a1 = {du, F, true};
        q.b1 = {w_up, C, false};
        q.out = dx; q.ldo = C;
        e = launch_simt(q, dtype, st);
    }
    if (want_dw) {
        Product q;
        q.M = (int)F; q.N = (int)C; q.K = (int)R;
        q.b0 = {x, C, false};
        q.ldo = C;
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            q.a0 = {i ? du : dg, F, false};
            q.out = i ? dw_up : dw_gate;
            e = launch_simt(q, dtype, st);
        }
        q.M = (int)C; q.N = (int)F;
        q.a0 = {dy, C, false};
        q.b0 = {at(saved, kept.h), F, false};
        q.out = dw_down; q.ldo = F;
        if (e == cudaSuccess) e = launch_simt(q, dtype, st);
    }
    return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

}  // extern "C"
