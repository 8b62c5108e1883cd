// fp32 products of the gated feed-forward on the tensor cores.
//
// An fp32 operand is three bf16 planes, a = h + m + l (split_f32), and
//   a b = h h' + (h m' + m h' + m m' + h l' + l h') + (m l' + l m' + l l'),
// the last bracket left out: |m| <= 2^-7 |a| and |l| <= 2^-16 |a|, so that it is at
// most 2^-22 |a b|, and of either sign:
// six bf16 products for one of fp32, a twelfth of the CUDA cores' time for the
// same number of multiplications (8192 against 256 floating-point operations a
// clock and SM, over six). The products themselves are exact; what has to be kept
// small is the tensor cores' accumulation, which cuts rather than rounds: the large
// products h h' have an accumulator of their own, and every CHUNK_KB * 64 steps of
// K both accumulators are added, rounded to nearest, to fp32 sums in the epilogue
// warps' registers. A run of 16 MMA steps then errs by about 3e-7, and the sum of
// runs by no more.
//
// Otherwise the kernel is the 16-bit one with 128 x 128 tiles of single CTAs: a ring
// of shared-memory stages, each one plane of A and of B, three for a K block, whose
// six products need no more copies than three would (48 bytes of shared memory fill
// a clock and SM). 4096 rows, blocks of 1024 x 4096, forward and backward: 1.54 ms,
// 200 TFLOP/s of fp32 products.
#include "ffn_tc.cuh"

namespace im2win {
namespace ffn {
namespace {

constexpr int BN = 128;
constexpr int PLANES = 3;
constexpr int A_BYTES = ROWS * BK * 2, B_BYTES = BN * BK * 2, STAGE = A_BYTES + B_BYTES;
constexpr int STAGES = 6;
constexpr int STAGED = 32 * 9;  // floats of a warp's staged outputs
constexpr int SMEM = STAGE * STAGES + 1024;
constexpr int SMEM_STAGED = SMEM + EPI_WARPS * STAGED * 4;  // (only where needed: it takes from L1)
constexpr int CHUNK_KB = 4;  // K blocks of one run of the accumulators

struct F32Params {
    CUtensorMap a[2][PLANES], b[2][PLANES];
    int M, N, KB, segs, batch, tiles_m, tiles_n, tiles;  // as for the 16-bit products
    int a_rows, a_blocks, b_blocks;
    int act;
    void *out, *out2;
    float *kept;
    int64_t ldo, plane;
    int vec;  // 16-byte fp32 stores
    float *part;
    int64_t part_ld, part_step;
    int first;
    uint32_t *status;
    Groups groups;
    const float *scale;
    int table_at, rows_bound;
};

// 16 columns of a row of whole 16-byte vectors in fp32, `n` columns from here on (a multiple of 4).
__device__ __forceinline__ void store_f32(float *dst, const F2 (&v)[PAIRS], int n) {
#pragma unroll
    for (int i = 0; i < PAIRS / 2; ++i)
        if (4 * i < n) reinterpret_cast<ulonglong2 *>(dst)[i] = make_ulonglong2(v[2 * i].v, v[2 * i + 1].v);
}
// A warp's 16 columns of 32 rows into rows of any pitch, through its part of shared memory,
// so that neighbouring lanes store neighbouring columns. rows, n: valid rows and columns.
__device__ __forceinline__ void store_f32_staged(float *dst, int64_t ldo, const F2 (&v)[PAIRS], int rows, int n, float *stage) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            split(v[half * 4 + i], a, b);
            stage[lane * 9 + 2 * i] = a, stage[lane * 9 + 2 * i + 1] = b;
        }
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int row = it * 4 + lane / 8, c = lane % 8;
            if (row < rows && half * 8 + c < n) dst[row * ldo + half * 8 + c] = stage[row * 9 + c];
        }
    }
}

// 8 columns of a row in three planes, `n` of them valid (planes have 16-byte aligned rows).
__device__ __forceinline__ void store_planes8(uint16_t *dst, int64_t plane, const F2 *v, int n) {
    uint16_t h[8], m[8], l[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        split(v[i], a, b);
        split_f32(a, h[2 * i], m[2 * i], l[2 * i]);
        split_f32(b, h[2 * i + 1], m[2 * i + 1], l[2 * i + 1]);
    }
    auto word = [](const uint16_t *x, int i) { return (uint32_t)x[2 * i] | ((uint32_t)x[2 * i + 1] << 16); };
    const uint16_t *planes[PLANES] = {h, m, l};
#pragma unroll
    for (int q = 0; q < PLANES; ++q) {
        uint16_t *to = dst + q * plane;
        if (n >= 8) {
            *reinterpret_cast<uint4 *>(to) =
                make_uint4(word(planes[q], 0), word(planes[q], 1), word(planes[q], 2), word(planes[q], 3));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) to[i] = planes[q][i];
        }
    }
}

// g, u -> a = act(g) in g and u act'(g) in u, and h = a u; 4 columns.
__device__ __forceinline__ void gate4(int act, F2 *g, F2 *u, F2 *h) {
    with_act_device(act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x[2], y[2], a[2], d[2];
            split(g[i], x[0], x[1]);
            split(u[i], y[0], y[1]);
            act_both<decltype(kind)::value>(x[0], a[0], d[0]);
            act_both<decltype(kind)::value>(x[1], a[1], d[1]);
            h[i] = f2(a[0] * y[0], a[1] * y[1]);
            g[i] = f2(a[0], a[1]);
            u[i] = f2(y[0] * d[0], y[1] * d[1]);
        }
    });
}
__device__ __forceinline__ ulonglong2 words(const F2 *v) { return make_ulonglong2(v[0].v, v[1].v); }

// N (a multiple of 8) columns of row m (below m_end) from column n on, from their sums v (GATED: g,
// and u); none: the row's outputs are zero.
template <int EPI, int N>
__device__ __forceinline__ void finish(const F32Params &p, F2 *v, F2 *u, int m, int n, int m_end, bool none = false,
                                       float scale = 1.0f) {
    const int left = p.N - n;
    if (m >= m_end || left <= 0) return;
    const int64_t at = (int64_t)m * p.ldo + n;
    if (EPI == EPI_STORE) return;  // (store_f32)
    float *kept_a = p.kept, *kept_b = p.kept + kept_count_f32(p.M, p.N);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        if (8 * i >= left) break;
        F2 first[4], second[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            F2 *x = v + 4 * i + 2 * j;
            const int64_t k = kept_index_f32(m, n + 8 * i + 4 * j, p.N);
            const bool in = 8 * i + 4 * j < left;
            if (EPI == EPI_GATED) {
                F2 *y = u + 4 * i + 2 * j;
                gate4(p.act, x, y, first + 2 * j);
                if (p.kept && in) {
                    *reinterpret_cast<ulonglong2 *>(kept_a + k) = words(x);
                    *reinterpret_cast<ulonglong2 *>(kept_b + k) = words(y);
                }
                if (p.scale) second[2 * j] = mul2(first[2 * j], f2(scale)), second[2 * j + 1] = mul2(first[2 * j + 1], f2(scale));
            } else if (in) {
                x[0] = mul2(x[0], f2(scale)), x[1] = mul2(x[1], f2(scale));
                const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(kept_a + k);
                const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(kept_b + k);
                first[2 * j] = mul2(x[0], F2{b.x}), first[2 * j + 1] = mul2(x[1], F2{b.y});
                second[2 * j] = mul2(x[0], F2{a.x}), second[2 * j + 1] = mul2(x[1], F2{a.y});
            } else {
                first[2 * j] = first[2 * j + 1] = second[2 * j] = second[2 * j + 1] = f2(0.0f);
            }
        }
        if (none) {
#pragma unroll
            for (int j = 0; j < 4; ++j) first[j] = second[j] = f2(0.0f);
        }
        store_planes8(static_cast<uint16_t *>(p.out) + at + 8 * i, p.plane, first, left - 8 * i);
        if (EPI == EPI_DGATED || p.scale) store_planes8(static_cast<uint16_t *>(p.out2) + at + 8 * i, p.plane, second, left - 8 * i);
    }
}

template <bool AK, bool BKM, int EPI, bool GROUPED>
__global__ void __launch_bounds__(THREADS, 1) f32_product(const __grid_constant__ F32Params p) {
    extern __shared__ unsigned char dyn[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ alignas(8) uint64_t bars[2 * STAGES + 4];
    const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * STAGES;
    const uint32_t acc_full = empty + 8 * STAGES, acc_empty = acc_full + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Ctl ctl{&abort_flag, p.status};

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, EPI_WARPS);
        }
        fence_mbar_init();
    }
    // (as in the 16-bit kernel; here a call's first launch is the splitting)
    if (warp == 2) alloc_tmem<1>(smem_u32(&tmem_slot), 4 * BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    allow_dependents();
    grid_dependency_wait();
    const uint32_t tmem = tmem_slot;  // buffer i: the sums of h h' at 2 i BN, the others' BN further
    if (p.first && blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;

    const GroupTable table = group_table(dyn + p.table_at, p.groups.E);
    if (GROUPED) {  // (as in the 16-bit kernel)
        if (warp == 3) fill_group_table<!AK>(table, p, ROWS, lane);
        __syncthreads();
    }
    auto walk = [&] {
        if constexpr (GROUPED) return GroupWalk<!AK>(p, table, ROWS, blockIdx.x, gridDim.x);
        else return Walk(p, blockIdx.x, gridDim.x);
    }();
    Work w;
    if (warp == 0 && lane == 0) {
        // ---- copies
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        uint32_t a_bytes = AK ? p.a_rows * BK * 2 : (p.a_rows + 63) / 64 * 64 * BK * 2;
        while (ok && walk.next(w)) {
            const int m0 = w.tm * ROWS + (GROUPED && AK ? w.row0 : 0);
            const int a_copies = GROUPED && AK ? min(max((w.pad_end - m0) / 64, 0), 2) : 0;  // (as in the 16-bit kernel)
            if (GROUPED && AK) a_bytes = a_copies * 64 * BK * 2;
            for (int kb = w.k0; ok && kb < w.k1; ++kb) {
                const int seg = kb >= p.KB ? 1 : 0, k = (kb - seg * p.KB) * BK + (GROUPED && !AK ? w.row0 : 0);
#pragma unroll 1
                for (int q = 0; q < PLANES; ++q) {
                    if (!(ok = bar_wait(empty + 8 * s, phase ^ 1, ctl, SITE_STAGE_EMPTY))) break;
                    const uint32_t sa = base + s * STAGE, sb = sa + A_BYTES, bar = full + 8 * s;
                    mbar_arrive_expect_tx(bar, a_bytes + B_BYTES);
                    const CUtensorMap *ma = &p.a[seg | w.z][q], *mb = &p.b[seg | w.z][q];
                    if (GROUPED && AK) {
                        for (int i = 0; i < a_copies; ++i) tma_2d<1>(sa + i * 64 * BK * 2, ma, k, m0 + i * 64, bar);
                    } else if (AK) {
                        tma_2d<1>(sa, ma, k, m0, bar);
                    } else if (p.a_blocks) {
                        tma_3d<1>(sa, ma, 0, k, m0 / 64, bar);
                    } else {
                        for (int i = 0; i < p.a_rows; i += 64) tma_2d<1>(sa + i * BK * 2, ma, m0 + i, k, bar);
                    }
                    if (GROUPED && EPI == EPI_GATED) {
                        tma_3d<1>(sb, &p.b[0][q], k, w.tn * (BN / 2), w.e, bar);
                        tma_3d<1>(sb + B_BYTES / 2, &p.b[1][q], k, w.tn * (BN / 2), w.e, bar);
                    } else if (GROUPED && AK) {
                        if (BKM) {
                            tma_3d<1>(sb, mb, k, w.tn * BN, w.e, bar);
                        } else if (p.b_blocks) {
                            tma_4d<1>(sb, mb, 0, k, w.tn * (BN / 64), w.e, bar);
                        } else {
#pragma unroll
                            for (int i = 0; i < BN; i += 64) tma_3d<1>(sb + i * BK * 2, mb, w.tn * BN + i, k, w.e, bar);
                        }
                    } else if (EPI == EPI_GATED) {  // gate rows, then up rows of the same hidden channels
                        tma_2d<1>(sb, &p.b[0][q], k, w.tn * (BN / 2), bar);
                        tma_2d<1>(sb + B_BYTES / 2, &p.b[1][q], k, w.tn * (BN / 2), bar);
                    } else if (BKM) {
                        tma_2d<1>(sb, mb, k, w.tn * BN, bar);
                    } else if (p.b_blocks) {
                        tma_3d<1>(sb, mb, 0, k, w.tn * (BN / 64), bar);
                    } else {
#pragma unroll
                        for (int i = 0; i < BN; i += 64) tma_2d<1>(sb + i * BK * 2, mb, w.tn * BN + i, k, bar);
                    }
                    if (++s == STAGES) s = 0, phase ^= 1;
                }
            }
        }
        if (ok) ok = drain(empty, STAGES, s, phase, ctl, SITE_STAGE_EMPTY);
        if (!ok) let_end();
    } else if (warp == 1 && lane == 0) {
        // ---- MMAs
        int s = 0, n_run = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t idesc = make_idesc(true, ROWS, BN) | (AK ? 0u : 1u << 15) | (BKM ? 0u : 1u << 16);
        const uint64_t da = smem_desc(base, AK ? 16u : BK * 128u, 1024u) | (2ull << 61);
        const uint64_t db = smem_desc(base + A_BYTES, BKM ? 16u : BK * 128u, 1024u) | (2ull << 61);
        constexpr uint32_t step_a = (AK ? 32u : 2048u) >> 4, step_b = (BKM ? 32u : 2048u) >> 4;
        // one product of a K block: the plane of A in stage sa by the plane of B in stage sb
        auto product = [&](uint32_t d, int sa, int sb, bool add) {
            const uint64_t a = da + ((uint32_t)(sa * STAGE) >> 4), b = db + ((uint32_t)(sb * STAGE) >> 4);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) mma<1>(d, a + k * step_a, b + k * step_b, idesc, add || k > 0);
        };
        while (ok && walk.next(w)) {
            for (int kb = w.k0; ok && kb < w.k1; kb += CHUNK_KB, ++n_run) {
                const int buf = n_run & 1;
                if (!(ok = bar_wait(acc_empty + 8 * buf, ((n_run >> 1) & 1) ^ 1, ctl, SITE_ACC_EMPTY))) break;
                tc_fence_after();
                const uint32_t large = tmem + buf * 2 * BN, small = large + BN;
                for (int b = kb; b < min(kb + CHUNK_KB, w.k1); ++b) {
                    int st[PLANES];
                    for (int q = 0; q < PLANES; ++q) {
                        if (!(ok = bar_wait(full + 8 * s, phase, ctl, SITE_STAGE_FULL))) break;
                        tc_fence_after();
                        st[q] = s;
                        if (q == 0) {
                            product(large, st[0], st[0], b > kb);
                        } else if (q == 1) {
                            product(small, st[0], st[1], b > kb);
                            product(small, st[1], st[0], true);
                            product(small, st[1], st[1], true);
                        } else {
                            product(small, st[0], st[2], true);
                            product(small, st[2], st[0], true);
                        }
                        if (++s == STAGES) s = 0, phase ^= 1;
                    }
                    if (!ok) break;
                    for (int q = 0; q < PLANES; ++q) commit<1>(empty + 8 * st[q]);
                }
                if (ok) commit<1>(acc_full + 8 * buf);
            }
        }
        if (!ok) let_end();
    } else if (warp >= 4) {
        // ---- outputs: a warp for 32 rows and two chunks of columns (GATED: one of g and its u)
        const int q = warp & 3, share = (warp - 4) >> 2;
        const int c0 = EPI == EPI_GATED ? share * CHUNK : share * 2 * CHUNK;
        const int c1 = EPI == EPI_GATED ? BN / 2 + share * CHUNK : c0 + CHUNK;
        float *stage = reinterpret_cast<float *>(dyn + STAGES * STAGE + 1024) + (warp - 4) * STAGED;
        int n_run = 0;
        bool ok = true;
        while (ok && walk.next(w)) {
            F2 sum[2][PAIRS];
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) sum[0][i] = sum[1][i] = f2(0.0f);
            for (int kb = w.k0; kb < w.k1; kb += CHUNK_KB, ++n_run) {
                const int buf = n_run & 1;
                if (!(ok = warp_bar_wait(acc_full + 8 * buf, (n_run >> 1) & 1, ctl, SITE_ACC_FULL))) break;
                tc_fence_after();
                const uint32_t taddr = tmem + buf * 2 * BN + ((uint32_t)(q * 32) << 16);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t large[CHUNK], small[CHUNK];
                    load_chunk(taddr + (half ? c1 : c0), large);
                    load_chunk(taddr + BN + (half ? c1 : c0), small);
                    tmem_wait_ld();
                    if (half == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acc_empty + 8 * buf);
                    }
                    F2 x[PAIRS], y[PAIRS];
                    pairs_of(large, x);
                    pairs_of(small, y);
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) sum[half][i] = add2(sum[half][i], add2(x[i], y[i]));
                }
            }
            if (!ok) break;
            const int m = w.tm * ROWS + q * 32 + lane + (GROUPED && AK ? w.row0 : 0);
            const int m_end = !GROUPED || !AK ? p.M : EPI == EPI_STORE ? w.row_end : w.pad_end;
            const bool none = GROUPED && AK && m >= w.row_end;
            const float scale = !GROUPED ? 1.0f : EPI != EPI_STORE && p.scale && !none ? p.scale[m] : 0.0f;
            if (GROUPED ? p.part && !w.whole : p.part != nullptr) {
                float *dst = GROUPED ? p.part + (int64_t)(2 * blockIdx.x + w.slot) * ROWS * BN + part_index(q * 32 + lane, 0, BN)
                                     : p.part + w.slot * p.part_step + ((int64_t)w.z * p.M + m) * p.part_ld + (int64_t)w.tn * BN;
                if (GROUPED && m < m_end) {
#pragma unroll
                    for (int i = 0; i < PAIRS / 2; ++i) {
                        *reinterpret_cast<ulonglong2 *>(dst + (c0 + 4 * i) * 32) = words(sum[0] + 2 * i);
                        *reinterpret_cast<ulonglong2 *>(dst + (c1 + 4 * i) * 32) = words(sum[1] + 2 * i);
                    }
                } else if (m < m_end) {
                    store_f32(dst + c0, sum[0], CHUNK);
                    store_f32(dst + c1, sum[1], CHUNK);
                }
            } else if (EPI == EPI_STORE) {
                float *out = static_cast<float *>(w.z ? p.out2 : p.out);
                if (GROUPED && !AK) out += (int64_t)w.e * p.M * p.ldo;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int n = w.tn * BN + c0 + half * CHUNK;
                    if (n >= p.N) break;
                    if (!p.vec) store_f32_staged(out + (int64_t)(m - lane) * p.ldo + n, p.ldo, sum[half], m_end - (m - lane), p.N - n, stage);
                    else if (m < m_end) store_f32(out + (int64_t)m * p.ldo + n, sum[half], p.N - n);
                }
            } else if (EPI == EPI_GATED) {
                finish<EPI, CHUNK>(p, sum[0], sum[1], m, w.tn * (BN / 2) + c0, m_end, none, scale);
            } else {
                finish<EPI, CHUNK>(p, sum[0], nullptr, m, w.tn * BN + c0, m_end, none, scale);
                finish<EPI, CHUNK>(p, sum[1], nullptr, m, w.tn * BN + c1, m_end, none, scale);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) free_tmem<1>(tmem, 4 * BN);
}

// Eight columns of a row, `left` of them there.
__device__ __forceinline__ void store_octet(const F32Params &p, float *out, const F2 (&v)[4], int left) {
    if (p.vec && left >= 8) {
        reinterpret_cast<ulonglong2 *>(out)[0] = words(v);
        reinterpret_cast<ulonglong2 *>(out)[1] = words(v + 2);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a, b;
            split(v[i / 2], a, b);
            if (i < left) out[i] = i & 1 ? b : a;
        }
    }
}

// Adds the partial tiles of a streamed launch: one thread for eight output columns.
template <int EPI>
__global__ void __launch_bounds__(256) f32_join(const __grid_constant__ F32Params p, int units) {
    allow_dependents();
    grid_dependency_wait();
    constexpr int COLS = EPI == EPI_GATED ? BN / 2 : BN;
    int z, m, n, count;
    const float *src;
    if (!join_source<COLS, BN>(p, ROWS, units, z, m, n, count, src)) return;
    F2 v[4], u[4];
    add_partials<EPI == EPI_GATED, BN>(src, p.part_step, count, v, u);
    if (EPI == EPI_STORE) {
        store_octet(p, static_cast<float *>(z ? p.out2 : p.out) + (int64_t)m * p.ldo + n, v, p.N - n);
    } else {
        finish<EPI, 8>(p, v, u, m, n, p.M);
    }
}

// The same for a streamed launch over experts.
template <bool AK, int EPI>
__global__ void __launch_bounds__(256) f32_group_join(const __grid_constant__ F32Params p, int units) {
    constexpr int COLS = EPI == EPI_GATED ? BN / 2 : BN;
    extern __shared__ unsigned char dyn[];
    allow_dependents();
    grid_dependency_wait();
    const GroupTable table = group_table(dyn, p.groups.E);
    if (threadIdx.x < 32) fill_group_table<!AK>(table, p, ROWS, threadIdx.x);
    __syncthreads();
    if (!AK) zero_empty<float>(table, p.groups.E, p.out, p.batch == 2 ? p.out2 : nullptr, (int64_t)p.M * p.ldo);
    Work w;
    int unit, last;
    if (!group_join_source(GroupSpace<!AK>(p, table, ROWS), units, w, unit, last)) return;
    const int m_end = !AK ? p.M : EPI == EPI_STORE ? w.row_end : w.pad_end;
    for (int id = blockIdx.x % JOIN_SHARES * 256 + threadIdx.x; id < ROWS * COLS / 8; id += JOIN_SHARES * 256) {
        const int row = id % ROWS, col = id / ROWS * 8;
        const int m = w.tm * ROWS + row + (AK ? w.row0 : 0), n = w.tn * COLS + col;
        if (m >= m_end || n >= p.N) continue;
        F2 v[4], u[4];
        add_parts<EPI == EPI_GATED>(p.part, ROWS, BN, row, col, unit, last, v, u);
        const bool none = AK && m >= w.row_end;
        if (EPI == EPI_STORE) {
            float *out = static_cast<float *>(w.z ? p.out2 : p.out) + (AK ? 0 : (int64_t)w.e * p.M * p.ldo);
            store_octet(p, out + (int64_t)m * p.ldo + n, v, p.N - n);
        } else {
            finish<EPI, 8>(p, v, u, m, n, m_end, none, p.scale && !none ? p.scale[m] : 0.0f);
        }
    }
}

template <bool AK, bool BKM, int EPI, bool GROUPED>
cudaError_t launch_kind(F32Params &p, const TcPlan &pl, cudaStream_t st) {
    constexpr auto kernel = f32_product<AK, BKM, EPI, GROUPED>;
    // (a streamed launch over experts finishes whole tiles itself)
    p.table_at = EPI == EPI_STORE && !p.vec && (GROUPED || !p.part) ? SMEM_STAGED : SMEM;
    const int smem = p.table_at + (GROUPED ? group_table_bytes(p.groups.E) : 0);
    cudaError_t e = allow_smem<kernel>(SMEM_STAGED + (GROUPED ? group_table_bytes(MAX_EXPERTS) : 0));
    if (e != cudaSuccess) return e;
    e = launch_with(kernel, pl.units, THREADS, smem, 1, st, p);
    if (e != cudaSuccess || !p.part) return e;
    if constexpr (GROUPED) {
        return launch_with(f32_group_join<AK, EPI>, group_join_blocks(pl.units, !AK), 256, group_table_bytes(p.groups.E), 1, st, p, pl.units);
    } else {
        return launch_with(f32_join<EPI>, join_blocks(p), 256, 0, 1, st, p, pl.units);
    }
}

template <bool GROUPED>
cudaError_t launch_any(F32Params &p, const TcPlan &pl, const Product &d, cudaStream_t st) {
    if (d.epi == EPI_GATED) return launch_kind<true, true, EPI_GATED, GROUPED>(p, pl, st);
    if (d.epi == EPI_DGATED) return launch_kind<true, false, EPI_DGATED, GROUPED>(p, pl, st);
    if (!d.a0.k_major) return launch_kind<false, false, EPI_STORE, GROUPED>(p, pl, st);
    if (d.b0.k_major) return launch_kind<true, true, EPI_STORE, GROUPED>(p, pl, st);
    return launch_kind<true, false, EPI_STORE, GROUPED>(p, pl, st);
}

}  // namespace

// A K block is 24 MMAs of 64 clocks.
TcPlan plan_f32(const Product &d) {
    const double epi = d.epi == EPI_STORE ? 1 : 3;
    return d.groups.E ? plan_groups(d, 1, BN, 0.95, epi) : plan_tiles(d, 1, BN, 0.95, epi);
}

cudaError_t launch_f32(const Product &d, uint32_t *status, bool first, void *part, cudaStream_t st) {
    const TcPlan pl = plan_f32(d);
    F32Params p = {};
    p.M = d.M; p.N = d.N; p.KB = (d.K + BK - 1) / BK;
    const bool two = d.a1.p != nullptr;
    p.segs = d.epi != EPI_GATED && two && !d.batch ? 2 : 1;
    p.batch = d.batch ? 2 : 1;
    p.tiles_m = pl.tiles_m; p.tiles_n = pl.tiles_n; p.tiles = p.batch * pl.tiles_m * pl.tiles_n;
    p.groups = d.groups;
    p.scale = d.scale;
    p.rows_bound = d.a0.k_major ? d.M : d.K;
    const int stack = d.a0.k_major ? d.groups.E : 0;
    if (d.groups.E && !d.a0.k_major) p.tiles *= d.groups.E;
    p.a_rows = std::min(ROWS, (d.M + 7) / 8 * 8);
    if (stack) p.a_rows = 64;  // (of one copy)
    p.a_blocks = !d.a0.k_major && d.M % 64 == 0;
    p.b_blocks = !d.b0.k_major && d.N % 64 == 0;
    const int b_box = d.epi == EPI_GATED ? BN / 2 : BN;
    for (int q = 0; q < PLANES; ++q) {
        if (!encode(p.a[0][q], d.a0, q, d.M, d.K, p.a_rows, p.a_blocks) ||
            !encode(p.b[0][q], d.b0, q, d.N, d.K, b_box, p.b_blocks, stack) ||
            (two && !encode(p.a[1][q], d.a1, q, d.M, d.K, p.a_rows, p.a_blocks)) ||
            (d.b1.p && !encode(p.b[1][q], d.b1, q, d.N, d.K, b_box, p.b_blocks, stack)))
            return cudaErrorInvalidValue;
    }
    p.act = d.act;
    p.out = d.out; p.out2 = d.out2; p.kept = static_cast<float *>(d.kept);
    p.ldo = d.ldo; p.plane = d.plane;
    p.vec = d.ldo % 4 == 0;
    if (pl.streamed) {
        p.part = static_cast<float *>(part);
        p.part_ld = pl.part_ld;
        p.part_step = pl.part_step;
    }
    p.status = status;
    p.first = first;
    return d.groups.E ? launch_any<true>(p, pl, d, st) : launch_any<false>(p, pl, d, st);
}

}  // namespace ffn
}  // namespace im2win
