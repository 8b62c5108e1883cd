// Gated feed-forward block: argument checks, buffers and the sequence of products.
#include <algorithm>
#include <initializer_list>

#include "gated_ffn.cuh"

using namespace im2win;
using namespace im2win::ffn;

namespace {

im2win_status check_dims(int64_t R, int64_t C, int64_t F, int dtype) {
    if (R < 0 || C < 1 || F < 1 || elem_size(dtype) == 0) return IM2WIN_ERR_INVALID_ARG;
    const int64_t most = 0x7fffffff - 1023, area = int64_t(1) << 40;
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

// A call's problem. The tensor cores' copies need row pitches that are multiples
// of 16 bytes: own buffers have such a pitch, and matrices of the caller whose
// width is no multiple of 8 are first copied to one. fp32 matrices are always
// copied, to three bf16 planes, and own ones are such planes.
struct Problem {
    int R, C, F, dtype, act;
    bool f32;
    int64_t Cp, Fp;  // pitches of rows of C and F elements
    Problem(int64_t R_, int64_t C_, int64_t F_, int act_, int dtype_)
        : R((int)R_), C((int)C_), F((int)F_), dtype(dtype_), act(act_), f32(dtype_ == IM2WIN_F32),
          Cp((C_ + 7) / 8 * 8), Fp((F_ + 7) / 8 * 8) {}

    // the forward pass of few rows has kernels of its own
    bool few() const { return is_few(R, C, F, dtype); }
    // own buffers
    size_t rows_c(int64_t rows) const { return (size_t)(rows * Cp) * (f32 ? 6 : 2); }
    size_t rows_f(int64_t rows) const { return (size_t)(rows * Fp) * (f32 ? 6 : 2); }
    bool copies(int64_t cols) const { return f32 || cols % 8 != 0; }

    Operand by_c(const void *p, int64_t rows, bool k_major) const { return {p, Cp, k_major, rows * Cp}; }
    Operand by_f(const void *p, int64_t rows, bool k_major) const { return {p, Fp, k_major, rows * Fp}; }

    Product gated(const void *x, const void *wg, const void *wu, void *h, void *kept) const {
        Product p;
        p.M = R; p.N = F; p.K = C;
        p.a0 = by_c(x, R, true); p.b0 = by_c(wg, F, true); p.b1 = by_c(wu, F, true);
        p.epi = EPI_GATED; p.act = act;
        p.out = h; p.ldo = Fp; p.plane = R * Fp; p.kept = kept;
        return p;
    }
    Product down(const void *h, const void *wd, void *y) const {
        Product p;
        p.M = R; p.N = C; p.K = F;
        p.a0 = by_f(h, R, true); p.b0 = by_f(wd, C, true);
        p.out = y; p.ldo = C;
        return p;
    }
    Product dgated(const void *dy, const void *wd, const void *kept, void *dg, void *du) const {
        Product p;
        p.M = R; p.N = F; p.K = C;
        p.a0 = by_c(dy, R, true); p.b0 = by_f(wd, C, false);
        p.epi = EPI_DGATED; p.act = act;
        p.out = dg; p.out2 = du; p.ldo = Fp; p.plane = R * Fp;
        p.kept = const_cast<void *>(kept);
        return p;
    }
    Product dx(const void *dg, const void *du, const void *wg, const void *wu, void *out) const {
        Product p;
        p.M = R; p.N = C; p.K = F;
        p.a0 = by_f(dg, R, true); p.b0 = by_c(wg, F, false);
        p.a1 = by_f(du, R, true); p.b1 = by_c(wu, F, false);
        p.out = out; p.ldo = C;
        return p;
    }
    Product dw_in(const void *dg, const void *du, const void *x, void *dwg, void *dwu) const {
        Product p;
        p.M = F; p.N = C; p.K = R;
        p.a0 = by_f(dg, R, false); p.a1 = by_f(du, R, false);
        p.b0 = p.b1 = by_c(x, R, false);
        p.batch = true;
        p.out = dwg; p.out2 = dwu; p.ldo = C;
        return p;
    }
    Product dw_down(const void *dy, const void *h, void *out) const {
        Product p;
        p.M = C; p.N = F; p.K = R;
        p.a0 = by_c(dy, R, false); p.b0 = by_f(h, R, false);
        p.out = out; p.ldo = F;
        return p;
    }
    // the forward pass that keeps nothing runs as one kernel
    bool fused() const;
    TcPlan plan(const Product &p) const { return f32 ? plan_f32(p) : plan_tc(p); }
};

// saved: h, then what the backward pass needs of g and u.
struct SavedParts {
    size_t h, kept, bytes;
    explicit SavedParts(const Problem &q) {
        Parts p(0);
        h = p.add(q.rows_f(q.R));
        kept = p.add(kept_bytes(q.R, q.F, q.f32));
        bytes = p.end;
    }
};

const void *const kSome = reinterpret_cast<const void *>(16);  // a present operand, where only sizes matter
void *const kSomeOut = reinterpret_cast<void *>(16);

bool Problem::fused() const {
    const double cost = f32 ? 0 : fused_cost(R, C, F);
    return cost > 0 && cost < plan(gated(kSome, kSome, kSome, kSomeOut, nullptr)).cost + plan(down(kSome, kSome, kSomeOut)).cost;
}

struct ForwardParts {
    bool one;  // the one kernel
    size_t h, h_lo, x, wg, wu, wd, part, bytes;
    ForwardParts(const Problem &q, bool saved) {
        Parts p(kStatusBytes);
        one = !saved && !q.few() && q.R > 0 && q.fused();
        if (q.few()) {  // fp32: h as it is; else its rounding (in `saved` if there is one) and the remainder
            h = p.add(q.f32 ? (size_t)q.R * q.F * 4 : saved ? 0 : q.rows_f(q.R));
            h_lo = p.add(q.f32 ? 0 : q.rows_f(q.R));
            x = wg = wu = wd = part = bytes = p.end;
            return;
        }
        h = h_lo = p.add(saved || one ? 0 : q.rows_f(q.R));
        x = p.add(q.copies(q.C) ? q.rows_c(q.R) : 0);
        wg = p.add(q.copies(q.C) ? q.rows_c(q.F) : 0);
        wu = p.add(q.copies(q.C) ? q.rows_c(q.F) : 0);
        wd = p.add(q.copies(q.F) ? q.rows_f(q.C) : 0);
        part = p.end;
        if (q.R > 0 && !one)
            p.add(std::max(q.plan(q.gated(kSome, kSome, kSome, kSomeOut, saved ? kSomeOut : nullptr)).part_bytes,
                           q.plan(q.down(kSome, kSome, kSomeOut)).part_bytes));
        bytes = p.end;
    }
};

struct BackwardParts {
    size_t dg, du, x, dy, wg, wu, wd, part, bytes;
    explicit BackwardParts(const Problem &q) {
        Parts p(kStatusBytes);
        dg = p.add(q.rows_f(q.R));
        du = p.add(q.rows_f(q.R));
        x = p.add(q.copies(q.C) ? q.rows_c(q.R) : 0);
        dy = p.add(q.copies(q.C) ? q.rows_c(q.R) : 0);
        wg = p.add(q.copies(q.C) ? q.rows_c(q.F) : 0);
        wu = p.add(q.copies(q.C) ? q.rows_c(q.F) : 0);
        wd = p.add(q.copies(q.F) ? q.rows_f(q.C) : 0);
        part = p.end;
        if (q.R > 0) {
            size_t most = 0;
            for (const Product &d : {q.dgated(kSome, kSome, nullptr, kSomeOut, kSomeOut),
                                     q.dx(kSome, kSome, kSome, kSome, kSomeOut),
                                     q.dw_in(kSome, kSome, kSome, kSomeOut, kSomeOut), q.dw_down(kSome, kSome, kSomeOut)})
                most = std::max(most, q.plan(d).part_bytes);
            p.add(most);
        }
        bytes = p.end;
    }
};

unsigned char *at(void *base, size_t off) { return static_cast<unsigned char *>(base) + off; }
const unsigned char *at(const void *base, size_t off) { return static_cast<const unsigned char *>(base) + off; }

bool known_act(int act) {
    return with_act(act, [](auto) {});
}

// The launches of one call, up to the first that fails.
struct Sequence {
    const Problem &q;
    void *ws;
    void *part;
    cudaStream_t st;
    cudaError_t e = cudaSuccess;
    bool cleared = false;
    Repitch copies[5];
    int n_copies = 0;

    // The matrix itself, or its copy at `to` that the products can read.
    const void *readable(const void *src, int rows, int cols, size_t to) {
        if (!q.copies(cols)) return src;
        copies[n_copies++] = {src, at(ws, to), rows, cols};
        return at(ws, to);
    }
    void copy() {
        if (n_copies && e == cudaSuccess) e = launch_repitch(copies, n_copies, q.f32, st);
    }
    void run(const Product &p) {
        if (e != cudaSuccess) return;
        uint32_t *status = static_cast<uint32_t *>(ws);
        e = q.f32 ? launch_f32(p, status, !cleared, part, st)
                  : launch_tc(p, q.dtype == IM2WIN_BF16, status, !cleared, part, st);
        cleared = true;
    }
};

}  // namespace

extern "C" {

im2win_status im2win_gated_ffn_size(int buffer, int64_t R, int64_t C, int64_t F, int dtype, size_t *bytes) {
    if (!bytes) return IM2WIN_ERR_INVALID_ARG;
    const im2win_status s = check_dims(R, C, F, dtype);
    if (s != IM2WIN_OK) return s;
    const Problem q(R, C, F, 0, dtype);
    switch (buffer) {
        case IM2WIN_FFN_FORWARD: *bytes = ForwardParts(q, false).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_TRAIN: *bytes = ForwardParts(q, true).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_BACKWARD: *bytes = BackwardParts(q).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_SAVED: *bytes = SavedParts(q).bytes; return IM2WIN_OK;
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
    const Problem q(R, C, F, act, dtype);
    const ForwardParts parts(q, saved != nullptr);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    const SavedParts own(q);
    void *h = saved ? at(saved, own.h) : at(ws, parts.h);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void *kept = saved ? at(saved, own.kept) : nullptr;
    if (q.few()) {
        const Few f = {q.R, q.C, q.F, act, x, w_gate, w_up, w_down, y, q.f32 ? at(ws, parts.h) : h,
                       at(ws, parts.h_lo), q.f32 ? (int64_t)q.F : q.Fp, static_cast<uint16_t *>(h), q.Fp, kept,
                       static_cast<uint32_t *>(ws)};
        return launch_few(f, dtype, st) == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
    }
    Sequence seq{q, ws, at(ws, parts.part), st};
    x = seq.readable(x, q.R, q.C, parts.x);
    w_gate = seq.readable(w_gate, q.F, q.C, parts.wg);
    w_up = seq.readable(w_up, q.F, q.C, parts.wu);
    w_down = seq.readable(w_down, q.C, q.F, parts.wd);
    seq.copy();
    if (parts.one) {
        const Fused f = {q.R, q.C, q.F, act, q.by_c(x, q.R, true), q.by_c(w_gate, q.F, true), q.by_c(w_up, q.F, true),
                         q.by_f(w_down, q.C, true), y};
        if (seq.e == cudaSuccess) seq.e = launch_fused(f, dtype == IM2WIN_BF16, static_cast<uint32_t *>(ws), st);
        return seq.e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
    }
    seq.run(q.gated(x, w_gate, w_up, h, kept));
    seq.run(q.down(h, w_down, y));
    return seq.e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (R == 0) {  // sums over no rows
        cudaError_t e = cudaSuccess;
        for (void *w : {dw_gate, dw_up, dw_down})
            if (w && e == cudaSuccess) e = cudaMemsetAsync(w, 0, (size_t)(C * F) * elem_size(dtype), st);
        return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
    }
    if (!dx && !want_dw) return IM2WIN_OK;
    const Problem q(R, C, F, act, dtype);
    const BackwardParts parts(q);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    const SavedParts own(q);
    void *dg = at(ws, parts.dg), *du = at(ws, parts.du);
    Sequence seq{q, ws, at(ws, parts.part), st};
    dy = seq.readable(dy, q.R, q.C, parts.dy);
    w_down = seq.readable(w_down, q.C, q.F, parts.wd);
    if (dx) {
        w_gate = seq.readable(w_gate, q.F, q.C, parts.wg);
        w_up = seq.readable(w_up, q.F, q.C, parts.wu);
    }
    if (want_dw) x = seq.readable(x, q.R, q.C, parts.x);
    seq.copy();
    seq.run(q.dgated(dy, w_down, at(saved, own.kept), dg, du));
    if (dx) seq.run(q.dx(dg, du, w_gate, w_up, dx));
    if (want_dw) {
        seq.run(q.dw_in(dg, du, x, dw_gate, dw_up));
        seq.run(q.dw_down(dy, at(saved, own.h), dw_down));
    }
    return seq.e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

}  // extern "C"
