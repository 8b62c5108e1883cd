// Gated feed-forward grouped by expert: argument checks, buffers and the sequence of launches.
//
//   plan, gather   rows to their experts: xs
//   gated          h = act(xs w_gate_e^T) * (xs w_up_e^T); training: hw = weight * h
//   down           ys = h w_down_e^T
//   combine        y = sum over a row's choices of weight * ys
// backward
//   gather         dy to the experts: dys; dweights = dy . ys
//   dgated         dh = weight * (dys w_down_e), made into dg, du
//   dx             dxs = dg w_gate_e + du w_up_e, summed over a row's choices
//   dw             dw_gate_e = dg^T xs, dw_up_e = du^T xs, dw_down_e = dys^T hw over the expert's rows
//
// The products are the gated feed-forward's kernels with the rows in groups. h, hw, dg and du are
// operands and rounded to the dtype, as there; ys and dxs stay in fp32 until a row's sum, and the
// weights are applied in fp32 before the rounding of hw, dg and du, so that no other rounding
// comes between the inputs and the outputs (16-bit ys, weight * dy and dxs made y 1.2 and dx
// 1.4 times as far off).
#include <algorithm>
#include <initializer_list>

#include "expert_ffn.cuh"

using namespace im2win;
using namespace im2win::ffn;

namespace {

im2win_status check_dims(int64_t T, int64_t k, int64_t E, int64_t C, int64_t F, int dtype) {
    if (T < 0 || k < 1 || E < 1 || C < 1 || F < 1 || elem_size(dtype) == 0) return IM2WIN_ERR_INVALID_ARG;
    const int64_t most = 0x7fffffff - 1023, area = int64_t(1) << 40;
    if (k > MAX_CHOICES || E > MAX_EXPERTS || T > (most - 64 * E) / k || C > most / E || F > most / E || C > area / F / E)
        return IM2WIN_ERR_UNSUPPORTED;
    const int64_t rows = grouped_rows(T * k, E);
    return rows > area / C || rows > area / F ? IM2WIN_ERR_UNSUPPORTED : IM2WIN_OK;
}

bool known_act(int act) {
    return with_act(act, [](auto) {});
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

struct Problem {
    int64_t T, rows, pairs;
    int k, E, C, F, dtype, act;
    bool f32;
    int64_t Cp, Fp;  // pitches of grouped rows and of copied weights
    Problem(int64_t T_, int64_t k_, int64_t E_, int64_t C_, int64_t F_, int act_, int dtype_)
        : T(T_), rows(grouped_rows(T_ * k_, E_)), pairs(T_ * k_), k((int)k_), E((int)E_), C((int)C_), F((int)F_), dtype(dtype_),
          act(act_), f32(dtype_ == IM2WIN_F32), Cp((C_ + 7) / 8 * 8), Fp((F_ + 7) / 8 * 8) {}

    // Inference of few pairs has kernels of its own. fp32, and widths whose experts' matrices would all be copied
    // to a pitch, up to 64 pairs (16 rows of 4 choices of 64 experts of 1000 x 1366: 97 us and 133 us; fp32, 4 rows
    // of 2 of 8 of 2048 x 4096: 122 us and 503 us). Else up to 8 pairs (4 rows of 2 of 8 of 2048 x 4096: 69 us
    // and 76 us), and up to 32 of smaller experts (16 rows of 2 of 8 of 1024 x 2048: 40 us and 46 us; of 2048 x
    // 4096: 111 us and 92 us; 32 rows of 1024 x 2048: 52 us and 46 us).
    bool few() const {
        if (f32 || copies(C) || copies(F)) return pairs <= FEW_PAIRS;
        return pairs <= 8 || (pairs <= 32 && (pairs < E ? pairs : E) * C * F <= (int64_t(1) << 25));
    }
    size_t operand(int64_t n, int64_t pitch) const { return (size_t)(n * pitch) * (f32 ? 6 : 2); }
    size_t result() const { return (size_t)(rows * Cp) * 4; }  // ys, dxs
    bool copies(int64_t cols) const { return f32 || cols % 8 != 0; }

    Operand rows_c(const void *p, bool k_major) const { return {p, Cp, k_major, rows * Cp}; }
    Operand rows_f(const void *p, bool k_major) const { return {p, Fp, k_major, rows * Fp}; }
    // the experts' matrices; the planes of copies of fp32 ones lie behind all of them
    Operand w_in(const void *p, bool k_major) const { return {p, Cp, k_major, (int64_t)E * F * Cp}; }
    Operand w_out(const void *p, bool k_major) const { return {p, Fp, k_major, (int64_t)E * C * Fp}; }

    Product product(int M, int N, int K) const {
        Product p;
        p.M = M; p.N = N; p.K = K;
        p.act = act;
        p.groups.E = E;
        p.rows = (double)pairs;
        return p;
    }
    Product gated(const void *xs, const void *wg, const void *wu, void *h, void *hw, void *kept) const {
        Product p = product((int)rows, F, C);
        p.a0 = rows_c(xs, true);
        p.b0 = w_in(wg, true), p.b1 = w_in(wu, true);
        p.epi = EPI_GATED;
        p.out = h, p.out2 = hw, p.ldo = Fp, p.plane = rows * Fp, p.kept = kept;
        return p;
    }
    Product down(const void *h, const void *wd, void *ys) const {
        Product p = product((int)rows, C, F);
        p.a0 = rows_f(h, true), p.b0 = w_out(wd, true);
        p.out = ys, p.ldo = Cp;
        return p;
    }
    Product dgated(const void *dys, const void *wd, void *kept, void *dg, void *du) const {
        Product p = product((int)rows, F, C);
        p.a0 = rows_c(dys, true), p.b0 = w_out(wd, false);
        p.epi = EPI_DGATED;
        p.out = dg, p.out2 = du, p.ldo = Fp, p.plane = rows * Fp, p.kept = kept;
        return p;
    }
    Product dx(const void *dg, const void *du, const void *wg, const void *wu, void *dxs) const {
        Product p = product((int)rows, C, F);
        p.a0 = rows_f(dg, true), p.b0 = w_in(wg, false);
        p.a1 = rows_f(du, true), p.b1 = w_in(wu, false);
        p.out = dxs, p.ldo = Cp;
        return p;
    }
    Product dw_in(const void *dg, const void *du, const void *xs, void *dwg, void *dwu) const {
        Product p = product(F, C, (int)rows);
        p.a0 = rows_f(dg, false), p.a1 = rows_f(du, false);
        p.b0 = p.b1 = rows_c(xs, false);
        p.batch = true;
        p.out = dwg, p.out2 = dwu, p.ldo = C;
        return p;
    }
    Product dw_down(const void *dys, const void *hw, void *out) const {
        Product p = product(C, F, (int)rows);
        p.a0 = rows_c(dys, false), p.b0 = rows_f(hw, false);
        p.out = out, p.ldo = F;
        return p;
    }
    size_t part_bytes(std::initializer_list<Product> list) const {
        size_t most = 0;
        for (const Product &p : list) most = std::max(most, (f32 ? plan_f32(p) : plan_tc(p)).part_bytes);
        return most;
    }
};

const void *const kSome = reinterpret_cast<const void *>(16);  // a present operand, where only sizes matter
void *const kSomeOut = reinterpret_cast<void *>(16);

struct SavedParts {
    size_t begin, count, slot, pair, scale, xs, h, hw, kept, ys, bytes;
    // keep: what the backward pass alone needs
    SavedParts(const Problem &q, size_t from, bool keep) {
        Parts p(from);
        begin = p.add((size_t)(q.E + 1) * 4);
        count = p.add((size_t)q.E * 4);
        slot = p.add((size_t)q.pairs * 4);
        pair = p.add((size_t)q.rows * 4);
        scale = p.add(keep ? (size_t)q.rows * 4 : 0);
        xs = p.add(q.operand(q.rows, q.Cp));
        h = p.add(q.operand(q.rows, q.Fp));
        hw = p.add(keep ? q.operand(q.rows, q.Fp) : 0);
        kept = p.add(keep ? kept_bytes(q.rows, q.F, q.f32) : 0);
        ys = p.add(q.result());
        bytes = p.end;
    }
};

// A forward call's workspace; without `saved`, its parts too.
struct ForwardParts {
    size_t hist, wg, wu, wd, part, own, h, h_lo, bytes;
    ForwardParts(const Problem &q, bool saved) {
        Parts p(kStatusBytes);
        h = p.add(q.few() && !saved ? (size_t)q.pairs * (q.f32 ? q.F * (size_t)4 : q.Fp * (size_t)2) : 0);
        h_lo = p.add(q.few() && !saved && !q.f32 ? (size_t)q.pairs * q.Fp * 2 : 0);
        if (q.few() && !saved) {
            hist = wg = wu = wd = part = own = bytes = p.end;
            return;
        }
        const int64_t per = pairs_per_block(q.pairs), blocks = (q.pairs + per - 1) / per;
        hist = p.add(blocks > 1 ? (size_t)blocks * q.E * 4 : 0);
        wg = p.add(q.copies(q.C) ? q.operand((int64_t)q.E * q.F, q.Cp) : 0);
        wu = p.add(q.copies(q.C) ? q.operand((int64_t)q.E * q.F, q.Cp) : 0);
        wd = p.add(q.copies(q.F) ? q.operand((int64_t)q.E * q.C, q.Fp) : 0);
        part = p.add(q.pairs == 0 ? 0 : q.part_bytes({q.gated(kSome, kSome, kSome, kSomeOut, nullptr, saved ? kSomeOut : nullptr),
                                                      q.down(kSome, kSome, kSomeOut)}));
        own = p.end;
        bytes = saved ? own : SavedParts(q, own, false).bytes;
    }
};

struct BackwardParts {
    size_t dys, scale, dg, du, dxs, wg, wu, wd, part, bytes;
    explicit BackwardParts(const Problem &q) {
        Parts p(kStatusBytes);
        dys = p.add(q.operand(q.rows, q.Cp));
        scale = p.add((size_t)q.rows * 4);
        dg = p.add(q.operand(q.rows, q.Fp));
        du = p.add(q.operand(q.rows, q.Fp));
        dxs = p.add(q.result());
        wg = p.add(q.copies(q.C) ? q.operand((int64_t)q.E * q.F, q.Cp) : 0);
        wu = p.add(q.copies(q.C) ? q.operand((int64_t)q.E * q.F, q.Cp) : 0);
        wd = p.add(q.copies(q.F) ? q.operand((int64_t)q.E * q.C, q.Fp) : 0);
        part = p.add(q.pairs == 0 ? 0 : q.part_bytes({q.dgated(kSome, kSome, kSomeOut, kSomeOut, kSomeOut),
                                                      q.dx(kSome, kSome, kSome, kSome, kSomeOut),
                                                      q.dw_in(kSome, kSome, kSome, kSomeOut, kSomeOut),
                                                      q.dw_down(kSome, kSome, kSomeOut)}));
        bytes = p.end;
    }
};

unsigned char *at(void *base, size_t off) { return static_cast<unsigned char *>(base) + off; }
int32_t *ints(void *base, size_t off) { return reinterpret_cast<int32_t *>(at(base, off)); }
float *floats(void *base, size_t off) { return reinterpret_cast<float *>(at(base, off)); }

Rows rows_of(const Problem &q, const SavedParts &s, void *saved) {
    return {q.T, q.rows, q.k, q.E, q.C, q.Cp, {ints(saved, s.begin), ints(saved, s.count), ints(saved, s.slot), ints(saved, s.pair)}};
}

// The launches of one call, up to the first that fails.
struct Sequence {
    const Problem &q;
    const Rows &rows;
    void *ws;
    void *part;
    cudaStream_t st;
    cudaError_t e = cudaSuccess;
    Repitch copies[3];
    int n_copies = 0;

    const void *readable(const void *src, int rows, int cols, size_t to) {
        if (!q.copies(cols)) return src;
        copies[n_copies++] = {src, at(ws, to), rows, cols};
        return at(ws, to);
    }
    template <typename Fn>
    void step(Fn f) {
        if (e == cudaSuccess) e = f();
    }
    void copy() {
        if (n_copies) step([&] { return launch_repitch(copies, n_copies, q.f32, st); });
    }
    // scale: the rows' factors, where not null
    void run(Product p, const float *scale = nullptr) {
        uint32_t *status = static_cast<uint32_t *>(ws);
        p.groups.begin = rows.plan.begin, p.groups.count = rows.plan.count;
        p.scale = scale;
        step([&] {
            return q.f32 ? launch_f32(p, status, false, part, st) : launch_tc(p, q.dtype == IM2WIN_BF16, status, false, part, st);
        });
    }
};

}  // namespace

extern "C" {

im2win_status im2win_expert_ffn_size(int buffer, int64_t T, int64_t k, int64_t E, int64_t C, int64_t F, int dtype,
                                     size_t *bytes) {
    if (!bytes) return IM2WIN_ERR_INVALID_ARG;
    const im2win_status s = check_dims(T, k, E, C, F, dtype);
    if (s != IM2WIN_OK) return s;
    const Problem q(T, k, E, C, F, 0, dtype);
    switch (buffer) {
        case IM2WIN_FFN_FORWARD: *bytes = ForwardParts(q, false).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_TRAIN: *bytes = ForwardParts(q, true).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_BACKWARD: *bytes = BackwardParts(q).bytes; return IM2WIN_OK;
        case IM2WIN_FFN_SAVED: *bytes = SavedParts(q, 0, true).bytes; return IM2WIN_OK;
        default: return IM2WIN_ERR_INVALID_ARG;
    }
}

im2win_status im2win_expert_ffn(const void *x, const int32_t *experts, const void *weights, const void *w_gate,
                                const void *w_up, const void *w_down, void *y, void *saved, void *ws, size_t ws_bytes,
                                int64_t T, int64_t k, int64_t E, int64_t C, int64_t F, int act, int dtype, void *stream) {
    const im2win_status s = check_dims(T, k, E, C, F, dtype);
    if (s != IM2WIN_OK) return s;
    if (!known_act(act)) return IM2WIN_ERR_INVALID_ARG;
    if (T == 0) return IM2WIN_OK;  // no rows: nothing to read or write
    if (!x || !experts || !weights || !w_gate || !w_up || !w_down || !y) return IM2WIN_ERR_INVALID_ARG;
    for (const void *p : {x, w_gate, w_up, w_down, (const void *)y, (const void *)saved, (const void *)ws})
        if (!aligned_to(p, 16)) return IM2WIN_ERR_MISALIGNED;
    if (!aligned_to(experts, 4) || !aligned_to(weights, elem_size(dtype))) return IM2WIN_ERR_MISALIGNED;
    const Problem q(T, k, E, C, F, act, dtype);
    const ForwardParts parts(q, saved != nullptr);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (q.few() && !saved) {
        const ExpertFew f = {(int)T, q.k, q.E, q.C, q.F, act, x, weights, w_gate, w_up, w_down, experts, y, at(ws, parts.h),
                             at(ws, parts.h_lo), q.f32 ? (int64_t)q.F : q.Fp, static_cast<uint32_t *>(ws)};
        return launch_expert_few(f, dtype, st) == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
    }
    const SavedParts own(q, saved ? 0 : parts.own, saved != nullptr);
    void *keep = saved ? saved : ws;
    const Rows rows = rows_of(q, own, keep);
    Sequence seq{q, rows, ws, at(ws, parts.part), st};
    seq.step([&] { return launch_plan(rows, experts, ints(ws, parts.hist), static_cast<uint32_t *>(ws), st); });
    w_gate = seq.readable(w_gate, q.E * q.F, q.C, parts.wg);
    w_up = seq.readable(w_up, q.E * q.F, q.C, parts.wu);
    w_down = seq.readable(w_down, q.E * q.C, q.F, parts.wd);
    seq.copy();
    seq.step([&] { return launch_gather(rows, x, weights, at(keep, own.xs), saved ? floats(keep, own.scale) : nullptr, dtype, st); });

    seq.run(q.gated(at(keep, own.xs), w_gate, w_up, at(keep, own.h), saved ? at(keep, own.hw) : nullptr,
                    saved ? at(keep, own.kept) : nullptr),
            saved ? floats(keep, own.scale) : nullptr);
    seq.run(q.down(at(keep, own.h), w_down, at(keep, own.ys)));
    seq.step([&] { return launch_combine(rows, floats(keep, own.ys), weights, y, dtype, st); });
    return seq.e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

im2win_status im2win_expert_ffn_backward(const void *dy, const void *weights, const void *w_gate, const void *w_up,
                                         const void *w_down, const void *saved, void *dx, void *dweights,
                                         void *dw_gate, void *dw_up, void *dw_down, void *ws, size_t ws_bytes,
                                         int64_t T, int64_t k, int64_t E, int64_t C, int64_t F, int act, int dtype,
                                         void *stream) {
    const im2win_status s = check_dims(T, k, E, C, F, dtype);
    if (s != IM2WIN_OK) return s;
    if (!known_act(act)) return IM2WIN_ERR_INVALID_ARG;
    const bool want_dw = dw_gate != nullptr;
    if ((dw_up != nullptr) != want_dw || (dw_down != nullptr) != want_dw) return IM2WIN_ERR_INVALID_ARG;
    if (T > 0 && (!dy || !weights || !w_gate || !w_up || !w_down || !saved)) return IM2WIN_ERR_INVALID_ARG;
    for (const void *p : {dy, w_gate, w_up, w_down, saved, (const void *)dx, (const void *)dw_gate, (const void *)dw_up,
                          (const void *)dw_down, (const void *)ws})
        if (!aligned_to(p, 16)) return IM2WIN_ERR_MISALIGNED;
    if (!aligned_to(weights, elem_size(dtype)) || !aligned_to(dweights, elem_size(dtype))) return IM2WIN_ERR_MISALIGNED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {  // sums over no rows
        cudaError_t e = cudaSuccess;
        for (void *w : {dw_gate, dw_up, dw_down})
            if (w && e == cudaSuccess) e = cudaMemsetAsync(w, 0, (size_t)(E * C * F) * elem_size(dtype), st);
        return e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
    }
    if (!dx && !dweights && !want_dw) return IM2WIN_OK;
    const Problem q(T, k, E, C, F, act, dtype);
    const BackwardParts parts(q);
    if (!ws || ws_bytes < parts.bytes) return IM2WIN_ERR_WORKSPACE;
    const SavedParts own(q, 0, true);
    void *keep = const_cast<void *>(saved);
    const Rows rows = rows_of(q, own, keep);
    Sequence seq{q, rows, ws, at(ws, parts.part), st};
    void *dys = at(ws, parts.dys), *dg = at(ws, parts.dg), *du = at(ws, parts.du);
    seq.step([&] {
        return launch_gather_back(rows, dy, weights, floats(keep, own.ys), dys, floats(ws, parts.scale), dweights,
                                  static_cast<uint32_t *>(ws), dtype, st);
    });
    if (dx || want_dw) {
        w_down = seq.readable(w_down, q.E * q.C, q.F, parts.wd);
        if (dx) {
            w_gate = seq.readable(w_gate, q.E * q.F, q.C, parts.wg);
            w_up = seq.readable(w_up, q.E * q.F, q.C, parts.wu);
        }
        seq.copy();
        seq.run(q.dgated(dys, w_down, at(keep, own.kept), dg, du), floats(ws, parts.scale));
    }
    if (dx) {
        seq.run(q.dx(dg, du, w_gate, w_up, at(ws, parts.dxs)));
        seq.step([&] { return launch_combine(rows, floats(ws, parts.dxs), nullptr, dx, dtype, st); });
    }
    if (want_dw) {
        seq.run(q.dw_in(dg, du, at(keep, own.xs), dw_gate, dw_up));
        seq.run(q.dw_down(dys, at(keep, own.hw), dw_down));
    }
    return seq.e == cudaSuccess ? IM2WIN_OK : IM2WIN_ERR_CUDA;
}

}  // extern "C"
