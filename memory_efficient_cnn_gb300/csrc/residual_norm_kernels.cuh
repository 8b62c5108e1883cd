// The norms around a residual block with its gate and residual scale:
//   r = res_scale * x + gate * post(y),  n = pre(r),  and the gradients.
//
// With m, i the mean (0 for RMS) and inverse deviation of a row v, its normed
// row is hat = (v - m) i and post(v) = hat * w + b; for a gradient d of post(v),
//   e = d * w,  dv = i (e - [mean(e)] - hat * mean(e * hat)),
// the bracket for LAYER only. dt = dr + pre'(dn) is the gradient of r.
#pragma once

#include "residual_norm.cuh"

namespace im2win {
namespace rnorm {

namespace {

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

// ---- rows in registers
//
// A row of at most TPR * EPT elements is held by TPR neighbouring threads, EPT
// fp32 values each, so that every input is read from memory once and the row's
// statistics are reductions over registers (two passes for LAYER: the second
// moment is taken about the mean). Thread t holds vectors t, t + TPR, ... of V
// elements: 16-byte vectors where C allows, else 4-byte ones, else elements.
// Arithmetic is on pairs of values (F2).

// Two neighbouring 16-bit values, as they lie in a word, and their fp32 pair.
__device__ __forceinline__ F2 pair_of_word(uint32_t w, bf16_t) {
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ F2 pair_of_word(uint32_t w, f16_t) {
    const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return f2(r.x, r.y);
}
__device__ __forceinline__ uint32_t word_of_pair(F2 v, bf16_t) {
    float a, b;
    split(v, a, b);
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t word_of_pair(F2 v, f16_t) {
    float a, b;
    split(v, a, b);
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}

template <typename T, int V, int EPT, int TPR>
struct Row {
    static constexpr int VPT = EPT / V, PAIRS = EPT / 2;
    using E = T;
    using P = Vec<T, V>;
    static constexpr bool WORDS = sizeof(T) == 2 && V >= 2;  // pairs of values are words
    struct Packed {
        P v[VPT];
    };
    static __device__ __forceinline__ int first(int j, int t) { return (j * TPR + t) * V; }
    static __device__ __forceinline__ bool inside(int e, int C, int t) { return first(e / V, t) < C; }
    // Columns past C (0 for a row that is not there) read as zero.
    static __device__ __forceinline__ void load(Packed &d, const void *p, int64_t at, int C, int t) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = first(j, t);
            if (c < C) {
                d.v[j] = *reinterpret_cast<const P *>(static_cast<const T *>(p) + at + c);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) d.v[j].v[i] = from_f32<T>(0.0f);
            }
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, int C, int t, const F2 (&v)[PAIRS]) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = first(j, t);
            if (c >= C) continue;
            P d;
            if constexpr (WORDS) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i)
                    reinterpret_cast<uint32_t *>(&d)[i] = word_of_pair(v[j * V / 2 + i], T());
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float a, b;
                    split(v[(j * V + i) / 2], a, b);
                    d.v[i] = from_f32<T>((j * V + i) % 2 ? b : a);
                }
            }
            *reinterpret_cast<P *>(static_cast<T *>(p) + at + c) = d;
        }
    }
    // Values 2 i and 2 i + 1.
    static __device__ __forceinline__ F2 pair(const Packed &d, int i) {
        if constexpr (WORDS) return pair_of_word(reinterpret_cast<const uint32_t *>(&d)[i], T());
        else return f2(to_f32(d.v[2 * i / V].v[2 * i % V]), to_f32(d.v[(2 * i + 1) / V].v[(2 * i + 1) % V]));
    }
    static __device__ __forceinline__ void clear_outside(F2 (&v)[PAIRS], int C, int t) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float a, b;
            split(v[i], a, b);
            v[i] = f2(inside(2 * i, C, t) ? a : 0.0f, inside(2 * i + 1, C, t) ? b : 0.0f);
        }
    }
};

// The rows a thread will need, copied ahead into its own part of shared memory
// (no barrier: nobody else reads it). Where a vector is too short for such copies:
// two arrays are loaded a row ahead into registers (the forward pass of 8382 x
// 2631 fp16 takes 86 us so, 93 us without), four when they are asked for.
template <typename R, int ARRAYS, int MOST, int THREADS>
struct Ahead {
    static constexpr bool ASYNC = sizeof(typename R::P) >= 4, REGS = !ASYNC && ARRAYS == 2;
    static constexpr int DEPTH = REGS ? 2 : MOST;
    static constexpr int BYTES = ASYNC ? DEPTH * ARRAYS * THREADS * (int)sizeof(typename R::Packed) : 0;
    unsigned char *base;
    int stage = 0;  // of the next row to be read
    typename R::Packed now[REGS ? ARRAYS : 1], later[REGS ? ARRAYS : 1];
    __device__ explicit Ahead(void *smem) : base(static_cast<unsigned char *>(smem)) {}
    // vectors of one stage and array: [VPT][THREADS], so that a warp's are consecutive
    __device__ __forceinline__ unsigned char *at(int s, int a, int j) {
        return base + ((size_t)((s * ARRAYS + a) * R::VPT + j) * THREADS + threadIdx.x) * sizeof(typename R::P);
    }
    // Starts the copies of a row (C = 0: zeros) into the stage `ahead` rows on; not
    // `wanted`: of none, as after the last row, whose stage may get other copies next.
    __device__ __forceinline__ void copy(int ahead, bool wanted, const void *const (&p)[ARRAYS], int64_t row_at, int C,
                                         int t) {
        if (REGS && wanted) {
#pragma unroll
            for (int a = 0; a < ARRAYS; ++a)
                if (p[a]) R::load(ahead == 0 ? now[a] : later[a], p[a], row_at, C, t);
        }
        if (!ASYNC) return;
        int s = stage + ahead;
        if (s >= DEPTH) s -= DEPTH;
#pragma unroll
        for (int a = 0; a < ARRAYS; ++a) {
            if (!p[a] || !wanted) continue;
#pragma unroll
            for (int j = 0; j < R::VPT; ++j) {
                const int c = R::first(j, t), bytes = c < C ? (int)sizeof(typename R::P) : 0;
                copy_vector(at(s, a, j), static_cast<const typename R::E *>(p[a]) + (bytes ? row_at + c : 0), bytes);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    static __device__ __forceinline__ void copy_vector(void *dst, const void *src, int bytes) {
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
        if (sizeof(typename R::P) == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
        else if (sizeof(typename R::P) == 8)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
    }
    // Waits until at most `later` rows started after this one are still on their way.
    template <int LATER>
    __device__ __forceinline__ void wait() {
        if (ASYNC) asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory");
    }
    __device__ __forceinline__ void read(typename R::Packed &d, int a, const void *p, int64_t row_at, int C, int t) {
        if (ASYNC) {
#pragma unroll
            for (int j = 0; j < R::VPT; ++j) d.v[j] = *reinterpret_cast<const typename R::P *>(at(stage, a, j));
        } else if (REGS) {
            d = now[a];
        } else {
            R::load(d, p, row_at, C, t);
        }
    }
    __device__ __forceinline__ void next() {
        if (++stage == DEPTH) stage = 0;
        if (REGS) {
#pragma unroll
            for (int a = 0; a < ARRAYS; ++a) now[a] = later[a];
        }
    }
};

// Parameters of C elements in shared memory, those that are given one after the
// other, as they are stored: a thread's part of one is a conflict-free access (the
// block's threads fill them together; the caller's barrier follows). Types of 4 bytes, whose copies
// would not fit beside the rows', read them through L1.
template <typename R, int ARRAYS, int TPR>
struct Params {
    static constexpr bool SHARED = sizeof(typename R::E) == 2;
    static constexpr int EACH = SHARED ? TPR * (int)sizeof(typename R::Packed) : 0, BYTES = ARRAYS * EACH;
    unsigned char *base;
    const void *const *from;
    int C, t, place[ARRAYS];
    __device__ Params(void *smem, const void *const *from_, int C_, int t_)
        : base(static_cast<unsigned char *>(smem)), from(from_), C(C_), t(t_) {
        int given = 0;
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i) place[i] = given, given += from[i] != nullptr;
        if (!SHARED || threadIdx.x >= TPR) return;
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i) {
            if (!from[i]) continue;
            typename R::Packed d;
            R::load(d, from[i], 0, C, t);
#pragma unroll
            for (int j = 0; j < R::VPT; ++j) at(i, j) = d.v[j];
        }
    }
    __device__ __forceinline__ typename R::P &at(int i, int j) {
        return reinterpret_cast<typename R::P *>(base)[(place[i] * R::VPT + j) * TPR + t];
    }
    __device__ __forceinline__ void read(typename R::Packed &d, int i) {
        if (SHARED) {
#pragma unroll
            for (int j = 0; j < R::VPT; ++j) d.v[j] = at(i, j);
        } else {
            R::load(d, from[i], 0, C, t);
        }
    }
};
enum Param { PAR_SCALE, PAR_W_POST, PAR_B_POST, PAR_W_PRE, PAR_B_PRE, PARAMS };

// Sums over the TPR threads of a row, the same bits in every one of them. Rows of
// more than a warp join their warps' sums through shared memory, in two buffers
// in turn: a buffer is written again only after the barrier of the reduction
// between, which every thread reaches after reading it.
template <int TPR, int THREADS>
struct RowReduce {
    static constexpr int LANES = TPR > 32 ? 32 : TPR, WARPS = TPR > 32 ? TPR / 32 : 1;
    float (*buf)[2][THREADS / 32];  // [2][2][THREADS / 32]
    int phase = 0;
    __device__ explicit RowReduce(float (*b)[2][THREADS / 32]) : buf(b) {}
    __device__ __forceinline__ void barrier() {
        if (TPR == THREADS) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"((int)threadIdx.x / TPR + 1), "r"(TPR) : "memory");
    }
    __device__ __forceinline__ float sum(float a) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (TPR > 32) {
            const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w0 = threadIdx.x / TPR * WARPS;
            if (lane == 0) buf[phase][0][warp] = a;
            barrier();
            a = buf[phase][0][w0 + lane % WARPS];
#pragma unroll
            for (int o = WARPS / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
            phase ^= 1;
        }
        return a;
    }
    // Two sums: the lower half of the lanes goes on with a, the upper with b.
    __device__ __forceinline__ float2 sum2(float a, float b) {
        const int lane = threadIdx.x & 31;
        const bool up = (lane & (LANES / 2)) != 0;
        float v = up ? b : a;
        v += __shfl_xor_sync(0xffffffffu, up ? a : b, LANES / 2);
#pragma unroll
        for (int o = LANES / 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int row0 = lane & ~(LANES - 1);
        if (TPR <= 32)
            return make_float2(__shfl_sync(0xffffffffu, v, row0), __shfl_sync(0xffffffffu, v, row0 + LANES / 2));
        const int warp = threadIdx.x >> 5, w0 = threadIdx.x / TPR * WARPS;
        if ((lane & 15) == 0) buf[phase][lane >> 4][warp] = v;
        barrier();
        if (WARPS <= 16) {
            v = buf[phase][lane / WARPS & 1][w0 + lane % WARPS];
#pragma unroll
            for (int o = WARPS / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            a = __shfl_sync(0xffffffffu, v, 0), b = __shfl_sync(0xffffffffu, v, WARPS);
        } else {
            a = buf[phase][0][lane], b = buf[phase][1][lane];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                b += __shfl_xor_sync(0xffffffffu, b, o);
            }
        }
        phase ^= 1;
        return make_float2(a, b);
    }
};

__device__ __forceinline__ float total2(F2 v) {
    float a, b;
    split(v, a, b);
    return a + b;
}

// v -> its normed values, zero past C; i is the inverse deviation.
template <typename R, typename Red>
__device__ __forceinline__ void norm_values(int kind, F2 (&v)[R::PAIRS], int C, bool full, float inv_c, float eps, int t,
                                            Red &red, float &i) {
    i = 1.0f;
    if (kind == IM2WIN_NORM_NONE) return;
    F2 a = f2(0.0f);
    if (kind == IM2WIN_NORM_LAYER) {
#pragma unroll
        for (int e = 0; e < R::PAIRS; ++e) a = add2(a, v[e]);
        const F2 m = f2(-red.sum(total2(a)) * inv_c);
#pragma unroll
        for (int e = 0; e < R::PAIRS; ++e) v[e] = add2(v[e], m);
        if (!full) R::clear_outside(v, C, t);
        a = f2(0.0f);
    }
#pragma unroll
    for (int e = 0; e < R::PAIRS; ++e) a = fma2(v[e], v[e], a);
    i = rsqrtf(red.sum(total2(a)) * inv_c + eps);  // (2 ulp at most; a division and a root took 40 instructions)
    const F2 ii = f2(i);
#pragma unroll
    for (int e = 0; e < R::PAIRS; ++e) v[e] = mul2(v[e], ii);
}

// One row a TPR threads; a block takes a run of rows, its row slots in turn.
// Two rows read, two written: the parameters stay in shared memory as they are
// stored, the next rows are on their way while one is worked on. Three blocks an SM
// where shared memory has room: 8192 rows of 4096 bf16 take 50 us, 5.4 TB/s (56 us in
// two); 200704 rows of 128 fp16 with two LAYER norms 44 us, 4.6 TB/s, half of the issue
// slots taken (38 instructions a value).
template <typename T, int V, int EPT, int TPR, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : 3)
    norm_forward_rows(const __grid_constant__ NormArgs p, const __grid_constant__ FastDiv per_gate) {
    using R = Row<T, V, EPT, TPR>;
    constexpr int RPB = THREADS / TPR;
    using A = Ahead<R, 2, 3, THREADS>;
    constexpr int DEPTH = A::DEPTH;
    extern __shared__ uint4 dyn[];
    __shared__ float buf[2][2][THREADS / 32];
    RowReduce<TPR, THREADS> red(buf);
    A ahead(dyn);
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR, C = (int)p.C;
    const bool full = C == TPR * EPT;
    const float inv_c = 1.0f / (float)C;
    const int64_t begin = p.R * blockIdx.x / gridDim.x, end = p.R * (blockIdx.x + 1) / gridDim.x;
    const int rounds = (int)((end - begin + RPB - 1) / RPB);
    const void *const rows[2] = {p.x, p.y};
    const void *const given[PARAMS] = {p.res_scale, p.w_post, p.b_post, p.w_pre, p.b_pre};
    auto start = [&](int k, int into) {
        const int64_t row = begin + (int64_t)k * RPB + slot;
        ahead.copy(into, k < rounds, rows, row * C, row < end ? C : 0, t);
    };
#pragma unroll
    for (int k = 0; k < DEPTH - 1; ++k) start(k, k);
    Params<R, PARAMS, TPR> par(reinterpret_cast<unsigned char *>(dyn) + A::BYTES, given, C, t);
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < rounds; ++k) {
        const int64_t row = begin + (int64_t)k * RPB + slot, at = row * C;
        const int width = row < end ? C : 0;
        start(k + DEPTH - 1, DEPTH - 1);
        ahead.template wait<DEPTH - 1>();
        typename R::Packed d, w;
        F2 r[R::PAIRS];
        float i;
        if (p.y) {
            typename R::Packed pg;
            if (p.gate) R::load(pg, p.gate, (int64_t)fdiv((uint32_t)row, per_gate) * C, width, t);
            ahead.read(d, 1, p.y, at, width, t);
#pragma unroll
            for (int e = 0; e < R::PAIRS; ++e) r[e] = R::pair(d, e);
            norm_values<R>(p.post, r, C, full, inv_c, p.eps, t, red, i);
            if (p.w_post) {
                par.read(w, PAR_W_POST);
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) r[e] = mul2(r[e], R::pair(w, e));
            }
            if (p.b_post) {
                par.read(w, PAR_B_POST);
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) r[e] = add2(r[e], R::pair(w, e));
            }
            if (p.gate) {
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) r[e] = mul2(r[e], R::pair(pg, e));
            }
        } else {
#pragma unroll
            for (int e = 0; e < R::PAIRS; ++e) r[e] = f2(0.0f);
        }
        ahead.read(d, 0, p.x, at, width, t);
        ahead.next();
        if (p.res_scale) {
            par.read(w, PAR_SCALE);
#pragma unroll
            for (int e = 0; e < R::PAIRS; ++e) r[e] = fma2(R::pair(d, e), R::pair(w, e), r[e]);
        } else {
#pragma unroll
            for (int e = 0; e < R::PAIRS; ++e) r[e] = add2(R::pair(d, e), r[e]);
        }
        if (p.r) R::store(p.r, at, width, t, r);
        if (p.n) {
            norm_values<R>(p.pre, r, C, full, inv_c, p.eps, t, red, i);
            if (p.w_pre) {
                par.read(w, PAR_W_PRE);
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) r[e] = mul2(r[e], R::pair(w, e));
            }
            if (p.b_pre) {
                par.read(w, PAR_B_PRE);
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) r[e] = add2(r[e], R::pair(w, e));
            }
            R::store(p.n, at, width, t, r);
        }
    }
}

// ---- the backward pass in one reading of its inputs
//
// A block walks rows and keeps the sums over them in registers, a thread for its
// own columns. Within a gate group dw_post, db_post and dgate all follow from
//   A = sum dt * yhat,  B = sum dt:   dgate = w A + b B,  dw_post += gate A,  db_post += gate B,
// so five sums are enough: A, B, sum x dt, sum dn rhat and sum dn (B and the last
// only where there is a bias). Two ways of cutting the rows:
//  long groups   block k takes rows [R k / blocks, R (k+1) / blocks), its row slots
//                in turn; at the end of a group and of its rows it joins its slots'
//                A and B into segment k + g (unique along the staircase of blocks and
//                groups) for dgate, and weighed with the gate into its sums;
//  short groups  a row slot takes whole groups, writes their dgate and adds the
//                weighed A and B to its sums in shared memory.
// Four rows read, two written. 8192 rows of 4096 bf16, RMS: 118 us; 200704 rows of 128
// fp16, LAYER: 86 us; instructions bound both (74 a value, half of the issue slots). One
// block an SM: five sums and a row's values take 124 registers of 128. Rows of 4097 to
// 8192 elements have 16 a thread, and part of the sums in local memory: 4096 rows of
// 8192 bf16, RMS, 159 us with one gate.
// Rows on their way, the one at hand among them: as many as leave shared memory for the rest.
template <typename R, bool SHORT>
constexpr int BACK_DEPTH = sizeof(typename R::Packed) <= 16                                          ? 3
                           : sizeof(typename R::Packed) <= 32 && !(SHORT && sizeof(typename R::E) == 2) ? 2
                                                                                                       : 1;
template <typename R, int THREADS, bool SHORT>
using BackAhead = Ahead<R, 4, BACK_DEPTH<R, SHORT>, THREADS>;
// Shared memory of the rows on their way, which also joins slots: THREADS * EPT floats.
template <typename R, int THREADS, bool SHORT>
constexpr int BACK_ROWS_BYTES = BackAhead<R, THREADS, SHORT>::BYTES > THREADS * R::PAIRS * 8 ? BackAhead<R, THREADS, SHORT>::BYTES
                                                                                         : THREADS * R::PAIRS * 8;

template <typename T, int V, int EPT, int TPR, int THREADS, bool SHORT>
__global__ void __launch_bounds__(THREADS, 1)
    norm_backward_fused(const __grid_constant__ NormArgs p, const __grid_constant__ BackPlan plan, float *part, float *seg,
                        T *dgate) {
    using R = Row<T, V, EPT, TPR>;
    using A = BackAhead<R, THREADS, SHORT>;
    constexpr int RPB = THREADS / TPR, DEPTH = BACK_DEPTH<R, SHORT>;
    constexpr int W = TPR * EPT;  // columns a slot holds
    // rows on their way, between groups [RPB][W] to join slots; parameters; SHORT: A and B weighed, [2][RPB][W]
    extern __shared__ uint4 dyn[];
    unsigned char *par_at = reinterpret_cast<unsigned char *>(dyn) + BACK_ROWS_BYTES<R, THREADS, SHORT>;
    float *sums = reinterpret_cast<float *>(par_at + Params<R, PARAMS, TPR>::BYTES);
    __shared__ float buf[2][2][THREADS / 32];
    RowReduce<TPR, THREADS> red(buf);
    A ahead(dyn);
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR, C = (int)p.C;
    const bool full = C == W;
    const float inv_c = 1.0f / (float)C;
    float *fold = sums + (size_t)slot * W, *join = reinterpret_cast<float *>(dyn);
    const void *const inputs[4] = {p.x, p.y, p.dr, p.dn};
    const void *const given[PARAMS] = {p.res_scale, p.w_post, p.b_post, p.w_pre, p.b_pre};
    Params<R, PARAMS, TPR> par(par_at, given, C, t);
    __syncthreads();
    F2 acc[BACK_SUMS][R::PAIRS];
#pragma unroll
    for (int q = 0; q < BACK_SUMS; ++q)
#pragma unroll
        for (int e = 0; e < R::PAIRS; ++e) acc[q][e] = f2(0.0f);
    if (SHORT) {
#pragma unroll
        for (int e = 0; e < EPT; ++e) fold[e * TPR + t] = fold[RPB * W + e * TPR + t] = 0.0f;
    }

    // Rows first, first + step, ... before last, of group g; `rounds` is the same for all slots.
    auto rows = [&](int64_t g, int64_t first, int64_t last, int step, int rounds, typename R::Packed &pg) {
        auto start = [&](int k, int into) {
            const int64_t row = first + (int64_t)k * step;
            ahead.copy(into, k < rounds, inputs, row * C, row < last ? C : 0, t);
        };
#pragma unroll
        for (int k = 0; k < DEPTH - 1; ++k) start(k, k);
        if (p.gate) R::load(pg, p.gate, g * C, C, t);
#pragma unroll 1
        for (int k = 0; k < rounds; ++k) {
            const int64_t row = first + (int64_t)k * step, at = row * C;
            const int width = row < last ? C : 0;
            const float eps = row < last ? p.eps : 1.0f;  // (a slot without a row: zeros throughout)
            start(k + DEPTH - 1, DEPTH - 1);
            ahead.template wait<DEPTH - 1>();
            F2 yh[R::PAIRS], rh[R::PAIRS], d[R::PAIRS];
            float iy = 1.0f, ir = 1.0f;
            typename R::Packed v, w;
            ahead.read(v, 0, p.x, at, width, t);
            if (p.res_scale) {
                par.read(w, PAR_SCALE);
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) rh[e] = mul2(R::pair(v, e), R::pair(w, e));
            } else {
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) rh[e] = R::pair(v, e);
            }
            if (p.y) {
                ahead.read(v, 1, p.y, at, width, t);
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) yh[e] = R::pair(v, e);
                norm_values<R>(p.post, yh, C, full, inv_c, eps, t, red, iy);
                if (p.dn) {
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) d[e] = yh[e];
                    if (p.w_post) {
                        par.read(w, PAR_W_POST);
#pragma unroll
                        for (int e = 0; e < R::PAIRS; ++e) d[e] = mul2(d[e], R::pair(w, e));
                    }
                    if (p.b_post) {
                        par.read(w, PAR_B_POST);
#pragma unroll
                        for (int e = 0; e < R::PAIRS; ++e) d[e] = add2(d[e], R::pair(w, e));
                    }
                    if (p.gate) {
#pragma unroll
                        for (int e = 0; e < R::PAIRS; ++e) d[e] = mul2(d[e], R::pair(pg, e));
                    }
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) rh[e] = add2(rh[e], d[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) yh[e] = f2(0.0f);
            }
            if (p.dr) {
                ahead.read(v, 2, p.dr, at, width, t);
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) d[e] = R::pair(v, e);
            } else {
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) d[e] = f2(0.0f);
            }
            if (p.dn) {
                norm_values<R>(p.pre, rh, C, full, inv_c, eps, t, red, ir);
                ahead.read(v, 3, p.dn, at, width, t);
                F2 n[R::PAIRS], e1 = f2(0.0f), e2 = f2(0.0f);
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) {
                    n[e] = R::pair(v, e);
                    acc[BACK_W_PRE][e] = fma2(n[e], rh[e], acc[BACK_W_PRE][e]);
                }
                if (p.b_pre) {
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) acc[BACK_B_PRE][e] = add2(acc[BACK_B_PRE][e], n[e]);
                }
                if (p.w_pre) {
                    par.read(w, PAR_W_PRE);
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) n[e] = mul2(n[e], R::pair(w, e));
                }
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) e2 = fma2(n[e], rh[e], e2);
                const F2 scale = f2(ir);
                if (p.pre == IM2WIN_NORM_LAYER) {
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) e1 = add2(e1, n[e]);
                    const float2 m = red.sum2(total2(e1), total2(e2));
                    e1 = f2(-m.x * inv_c), e2 = f2(-m.y * inv_c);
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) d[e] = fma2(fma2(rh[e], e2, add2(n[e], e1)), scale, d[e]);
                    if (!full) R::clear_outside(d, C, t);
                } else {
                    e2 = f2(-red.sum(total2(e2)) * inv_c);
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) d[e] = fma2(fma2(rh[e], e2, n[e]), scale, d[e]);
                }
            }
            // d is dt, zero past C and in a slot without a row
            ahead.read(v, 0, p.x, at, width, t);
            ahead.next();
#pragma unroll
            for (int e = 0; e < R::PAIRS; ++e) {
                acc[BACK_RES][e] = fma2(R::pair(v, e), d[e], acc[BACK_RES][e]);
                acc[BACK_A][e] = fma2(d[e], yh[e], acc[BACK_A][e]);
            }
            if (p.b_post) {
#pragma unroll
                for (int e = 0; e < R::PAIRS; ++e) acc[BACK_B][e] = add2(acc[BACK_B][e], d[e]);
            }
            if (p.dx) {
                if (p.res_scale) {
                    par.read(w, PAR_SCALE);
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) rh[e] = mul2(d[e], R::pair(w, e));
                    R::store(p.dx, at, width, t, rh);
                } else {
                    R::store(p.dx, at, width, t, d);
                }
            }
            if (p.dy) {
                if (p.gate) {
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) d[e] = mul2(d[e], R::pair(pg, e));
                }
                if (p.w_post) {
                    par.read(w, PAR_W_POST);
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) d[e] = mul2(d[e], R::pair(w, e));
                }
                if (p.post != IM2WIN_NORM_NONE) {
                    F2 f1 = f2(0.0f), s2 = f2(0.0f);
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) s2 = fma2(d[e], yh[e], s2);
                    if (p.post == IM2WIN_NORM_LAYER) {
#pragma unroll
                        for (int e = 0; e < R::PAIRS; ++e) f1 = add2(f1, d[e]);
                        const float2 m = red.sum2(total2(f1), total2(s2));
                        f1 = f2(-m.x * inv_c), s2 = f2(-m.y * inv_c);
#pragma unroll
                        for (int e = 0; e < R::PAIRS; ++e) d[e] = add2(d[e], f1);
                    } else {
                        s2 = f2(-red.sum(total2(s2)) * inv_c);
                    }
                    const F2 scale = f2(iy);
#pragma unroll
                    for (int e = 0; e < R::PAIRS; ++e) d[e] = mul2(fma2(yh[e], s2, d[e]), scale);
                }
                R::store(p.dy, at, width, t, d);
            }
        }
    };
    // Adds one sum over the block's slots, in their order, clears it and hands each column's to put.
    auto join_slots = [&](F2(&sum)[R::PAIRS], auto put) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            float a, b;
            split(sum[e / 2], a, b);
            join[slot * W + R::first(e / V, t) + e % V] = e % 2 ? b : a;
        }
#pragma unroll
        for (int e = 0; e < R::PAIRS; ++e) sum[e] = f2(0.0f);
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += THREADS) {
            float v = 0.0f;
#pragma unroll 8
            for (int i = 0; i < RPB; ++i) v += join[i * W + c];
            put(c, v);
        }
        __syncthreads();
    };
    auto put_part = [&](int q, F2(&sum)[R::PAIRS]) {
        float *dst = part + ((int64_t)q * gridDim.x + blockIdx.x) * C;
        join_slots(sum, [&](int c, float v) { dst[c] = v; });
    };

    typename R::Packed pg;
    if (SHORT) {
        // slot s of all takes groups s, s + slots, ...
        const int64_t slots = (int64_t)gridDim.x * RPB;
        for (int64_t g0 = (int64_t)blockIdx.x * RPB; g0 < plan.groups; g0 += slots) {
            const int64_t g = g0 + slot, first = g * p.per_gate;
            const int64_t last = g < plan.groups ? min(p.R, first + p.per_gate) : first;
            rows(g < plan.groups ? g : 0, first, last, 1, (int)p.per_gate, pg);
            if (!p.y || g >= plan.groups) continue;  // (a slot without a group has the first one's gate: nothing to weigh)
            typename R::Packed w, b;
            if (p.w_post) R::load(w, p.w_post, 0, C, t);
            if (p.b_post) R::load(b, p.b_post, 0, C, t);
            F2 d[R::PAIRS];
#pragma unroll
            for (int e = 0; e < R::PAIRS; ++e) {
                const F2 gate = p.gate ? R::pair(pg, e) : f2(1.0f);
                d[e] = p.w_post ? mul2(R::pair(w, e), acc[BACK_A][e]) : acc[BACK_A][e];
                if (p.b_post) d[e] = fma2(R::pair(b, e), acc[BACK_B][e], d[e]);
                float a0, a1, b0, b1;
                split(mul2(gate, acc[BACK_A][e]), a0, a1);
                split(mul2(gate, acc[BACK_B][e]), b0, b1);
                fold[2 * e * TPR + t] += a0, fold[(2 * e + 1) * TPR + t] += a1;
                fold[RPB * W + 2 * e * TPR + t] += b0, fold[RPB * W + (2 * e + 1) * TPR + t] += b1;
                acc[BACK_A][e] = acc[BACK_B][e] = f2(0.0f);
            }
            if (dgate) R::store(dgate, g * C, C, t, d);
        }
#pragma unroll
        for (int e = 0; e < R::PAIRS; ++e) {
            acc[BACK_A][e] = f2(fold[2 * e * TPR + t], fold[(2 * e + 1) * TPR + t]);
            acc[BACK_B][e] = f2(fold[RPB * W + 2 * e * TPR + t], fold[RPB * W + (2 * e + 1) * TPR + t]);
        }
        put_part(BACK_A, acc[BACK_A]);
        put_part(BACK_B, acc[BACK_B]);
    } else {
        const int64_t begin = p.R * blockIdx.x / gridDim.x, end = p.R * (blockIdx.x + 1) / gridDim.x;
        for (int64_t at = begin; at < end;) {
            const int64_t g = at / p.per_gate, last = min(end, (g + 1) * p.per_gate);
            rows(g, at + slot, last, RPB, (int)((last - at + RPB - 1) / RPB), pg);
            if (p.y) {
                for (int q = BACK_A; q <= BACK_B; ++q) {
                    float *dst = seg + ((blockIdx.x + g) * 2 + (q - BACK_A)) * C;
                    float *weighed = part + ((int64_t)q * gridDim.x + blockIdx.x) * C;
                    const bool new_sum = at == begin;
                    auto put = [&](int c, float v) {  // (the same thread for a column every time)
                        dst[c] = v;
                        v *= load_or<T>(p.gate, g * C + c, 1.0f);
                        weighed[c] = new_sum ? v : weighed[c] + v;
                    };
                    if (q == BACK_A) join_slots(acc[BACK_A], put);
                    else join_slots(acc[BACK_B], put);
                }
            }
            at = last;
        }
    }
    put_part(BACK_RES, acc[BACK_RES]);
    put_part(BACK_W_PRE, acc[BACK_W_PRE]);
    put_part(BACK_B_PRE, acc[BACK_B_PRE]);
}

// Joins the fused pass's partial sums: 32 columns a block, its 8 warps over the
// partials in turn, then the warps' in order. blockIdx.y: 0 dres_scale, 1 dw_pre,
// 2 db_pre, 3 dw_post, 4 db_post, then dgate of groups y - 5, y - 5 + (gridDim.y - 5), ...
// (long groups).
template <typename T>
__global__ void __launch_bounds__(256) norm_join(const __grid_constant__ NormArgs p, const __grid_constant__ BackPlan plan,
                                                 const float *part, const float *seg, JoinOuts o) {
    __shared__ float s[2][8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t C = p.C, c = (int64_t)blockIdx.x * 32 + lane, from = min(c, C - 1);
    const int what = blockIdx.y < BACK_SUMS ? (int)blockIdx.y : BACK_SUMS;
    T *out = static_cast<T *>(what < BACK_SUMS ? o.out[what] : o.dgate);
    if (!out) return;
    auto over_warps = [&](float a, float b) {
        s[0][warp][lane] = a, s[1][warp][lane] = b;
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a += s[0][i][lane], b += s[1][i][lane];
        __syncthreads();
        return make_float2(a, b);
    };
    if (what < BACK_SUMS) {
        const float *src = part + (int64_t)what * plan.blocks * C + from;
        float v = 0.0f;
#pragma unroll 8
        for (int k = warp; k < plan.blocks; k += 8) v += src[k * C];
        v = over_warps(v, 0.0f).x;
        if (warp == 0 && c < C) out[c] = from_f32<T>(v);
        return;
    }
    const int stride = gridDim.y - BACK_SUMS;
    for (int64_t g = blockIdx.y - BACK_SUMS; g < plan.groups; g += stride) {
        // the blocks whose rows meet the group's
        const int64_t lo = g * p.per_gate, hi = min(p.R, lo + p.per_gate);
        int k0 = (int)(lo * plan.blocks / p.R), k1 = (int)((hi - 1) * plan.blocks / p.R);
        while (k0 + 1 < plan.blocks && p.R * (k0 + 1) / plan.blocks <= lo) ++k0;
        while (k1 + 1 < plan.blocks && p.R * (k1 + 1) / plan.blocks < hi) ++k1;
        float a = 0.0f, b = 0.0f;
        const float *src = seg + 2 * g * C + from;
#pragma unroll 4
        for (int k = k0 + warp; k <= k1; k += 8) {
            a += src[2 * k * C];
            b += src[(2 * k + 1) * C];
        }
        const float2 v = over_warps(a, b);
        if (warp == 0 && c < C)
            out[g * C + c] = from_f32<T>(fmaf(load_or<T>(p.w_post, c, 1.0f), v.x, load_or<T>(p.b_post, c, 0.0f) * v.y));
    }
}

template <typename T, int V, int EPT, int TPR, bool SHORT>
cudaError_t launch_fused(const NormArgs &p, const BackPlan &plan, float *part, float *seg, T *dgate, cudaStream_t st) {
    constexpr int THREADS = FUSED_THREADS;
    using R = Row<T, V, EPT, TPR>;
    constexpr int smem = BACK_ROWS_BYTES<R, THREADS, SHORT> + Params<R, PARAMS, TPR>::BYTES + (SHORT ? 2 * THREADS * EPT * 4 : 0);
    static_assert(smem <= 226 * 1024, "a block's shared memory");
    auto kernel = norm_backward_fused<T, V, EPT, TPR, THREADS, SHORT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<plan.blocks, THREADS, smem, st>>>(p, plan, part, seg, dgate);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_fused_tpr(const NormArgs &p, const BackPlan &plan, float *part, float *seg, T *dgate, cudaStream_t st) {
    auto as = [&](auto ept, auto tpr) {
        constexpr int EPT = decltype(ept)::value, TPR = decltype(tpr)::value;
        return plan.short_groups ? launch_fused<T, V, EPT, TPR, true>(p, plan, part, seg, dgate, st)
                                 : launch_fused<T, V, EPT, TPR, false>(p, plan, part, seg, dgate, st);
    };
    if (plan.ept == 16) return as(IntC<16>(), IntC<512>());
    auto with = [&](auto tpr) { return as(IntC<8>(), tpr); };
    switch (plan.tpr) {
        case 8: return with(IntC<8>());
        case 16: return with(IntC<16>());
        case 32: return with(IntC<32>());
        case 64: return with(IntC<64>());
        case 128: return with(IntC<128>());
        case 256: return with(IntC<256>());
        default: return with(IntC<512>());
    }
}

// Elements of the widest vector that rows of C elements allow; calls f with it.
template <typename T, typename Fn>
inline cudaError_t with_vector(int64_t C, Fn f) {
    constexpr int wide = 16 / (int)sizeof(T), mid = 4 / (int)sizeof(T);
    return C % wide == 0 ? f(IntC<wide>()) : C % mid == 0 ? f(IntC<mid>()) : f(IntC<1>());
}

// 32 bytes of a row a thread.
template <typename T, int V, int TPR>
cudaError_t launch_rows(const NormArgs &p, cudaStream_t st) {
    constexpr int THREADS = TPR > 256 ? TPR : 256, RPB = THREADS / TPR, EPT = 32 / (int)sizeof(T);
    using R = Row<T, V, EPT, TPR>;
    auto kernel = norm_forward_rows<T, V, EPT, TPR, THREADS>;
    using Pars = Params<R, PARAMS, TPR>;
    constexpr int most = Ahead<R, 2, 3, THREADS>::BYTES + Pars::BYTES;
    if (most > 32 * 1024) {  // (48 KB with the static part need no leave)
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    int smem = most - Pars::BYTES;
    for (const void *given : {p.res_scale, p.w_post, p.b_post, p.w_pre, p.b_pre}) smem += given ? Pars::EACH : 0;
    // three blocks an SM where their shared memory fits (226 KB with the static part)
    const int per_sm = THREADS > 256 ? 1 : 3 * (smem + 2048) <= 226 * 1024 ? 3 : 2;
    const int64_t blocks = (p.R + RPB - 1) / RPB;
    const FastDiv per = make_fastdiv((uint32_t)std::min(p.per_gate, p.R));
    kernel<<<(unsigned)std::min<int64_t>(blocks, SMS * per_sm), THREADS, smem, st>>>(p, per);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_forward(const NormArgs &p, cudaStream_t st) {
    const int64_t threads = (p.C * (int64_t)sizeof(T) + 31) / 32;  // of a row
    if (threads <= 4) return launch_rows<T, V, 4>(p, st);
    if (threads <= 8) return launch_rows<T, V, 8>(p, st);
    if (threads <= 16) return launch_rows<T, V, 16>(p, st);
    if (threads <= 32) return launch_rows<T, V, 32>(p, st);
    if (threads <= 64) return launch_rows<T, V, 64>(p, st);
    if (threads <= 128) return launch_rows<T, V, 128>(p, st);
    if (threads <= 256) return launch_rows<T, V, 256>(p, st);
    if constexpr (sizeof(T) == 4)
        if (threads > 512) return launch_rows<T, V, 1024>(p, st);
    return launch_rows<T, V, 512>(p, st);
}

}  // namespace

template <typename T>
cudaError_t launch_norm_forward(const NormArgs &p, cudaStream_t st) {
    if (p.C <= 8 * 1024) return with_vector<T>(p.C, [&](auto v) { return launch_forward<T, decltype(v)::value>(p, st); });
    norm_forward<T><<<(unsigned)p.R, ROW_THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm_backward(const NormArgs &args, const ColumnGrads &g, void *ws, cudaStream_t st) {
    NormArgs p = args;
    const BackwardParts parts(p.R, p.C, p.per_gate);
    unsigned char *base = static_cast<unsigned char *>(ws);
    p.stats = reinterpret_cast<float *>(base + parts.stats);
    float *part = reinterpret_cast<float *>(base + parts.part), *seg = reinterpret_cast<float *>(base + parts.seg);
    T *dgate = static_cast<T *>(g.dgate);
    const BackPlan fused = plan_back(p.R, p.C, p.per_gate);
    if (fused.blocks) {
        const cudaError_t e = with_vector<T>(
            p.C, [&](auto v) { return launch_fused_tpr<T, decltype(v)::value>(p, fused, part, seg, dgate, st); });
        if (!g.any() || e != cudaSuccess) return e;
        const JoinOuts o = {{g.dres_scale, g.dw_pre, g.db_pre, g.dw_post, g.db_post}, fused.short_groups ? nullptr : g.dgate};
        const dim3 grid((unsigned)((p.C + 31) / 32),
                        BACK_SUMS + (o.dgate ? (unsigned)std::min<int64_t>(fused.groups, 1024) : 0));
        norm_join<T><<<grid, 256, 0, st>>>(p, fused, part, seg, o);
        return cudaGetLastError();
    }
    const SumPlan plan = plan_sums(p.R, p.per_gate);
    const int64_t col_blocks = (p.C + SUM_COLS - 1) / SUM_COLS;
    norm_backward_rows<T><<<(unsigned)p.R, ROW_THREADS, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (!g.any() || e != cudaSuccess) return e;
    norm_column_sums<T><<<(unsigned)(plan.tasks * col_blocks), SUM_COLS * SUM_LANES, 0, st>>>(p, plan, col_blocks, part, dgate);
    void *outs[SUMS] = {g.dres_scale, g.dw_post, g.db_post, g.dw_pre, g.db_pre, plan.group_splits > 1 ? g.dgate : nullptr};
    for (int q = 0; q < SUMS; ++q) {
        if (!outs[q]) continue;
        const int64_t total = q == SUM_GATE ? plan.groups * p.C : p.C;
        join_partials<T><<<(unsigned)((total + 255) / 256), 256, 0, st>>>(
            part + q * plan.tasks * p.C, q == SUM_GATE ? plan.group_splits : plan.tasks, total, p.C,
            static_cast<T *>(outs[q]));
    }
    return cudaGetLastError();
}

}  // namespace rnorm
}  // namespace im2win
