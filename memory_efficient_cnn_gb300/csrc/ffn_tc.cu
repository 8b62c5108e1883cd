// Products of the gated feed-forward on the tensor cores (fp16/bf16 operands,
// fp32 accumulators in tensor memory).
//
// One persistent warp-specialised kernel computes D = A B^T tile by tile: one
// thread issues TMA copies of 64 steps of K into a ring of shared-memory stages,
// one issues tcgen05.mma on them, sixteen warps turn finished accumulators into
// outputs while the next tile accumulates in the other half of tensor memory.
// Operands may be stored with K or with the output index innermost (the backward
// products read every matrix as it lies): both are 128-byte-swizzled layouts
// that the copies write and the MMA reads.
//
// Two tile shapes: pairs of CTAs (cta_group::2) share 256 x 256 tiles, each
// staging half of A and half of B (64 bytes of shared memory fill per clock and
// SM at the MMA's full rate: a single CTA's 128 x 128 tile needs twice that);
// single CTAs with 128 x 128 tiles serve outputs of few tiles. With fewer tiles
// than SMs, or a last wave that would leave most idle, the K steps of all tiles
// are dealt out evenly ("streamed"): a CTA takes a contiguous run of steps,
// which may begin and end inside a tile, and writes fp32 partial tiles, which a
// second kernel adds in the order of K.
//
// Large products run at 1570 to 1800 TFLOP/s (8192 rows, blocks of 4096 x 10240, under
// the power cap; the MMAs alone at 1930). Short K leaves the epilogue as the bound:
// 200704 x 512 of gelu over K = 128 take 102 us (21 instructions a value, issue slots
// 57% taken), the product back to 128 columns 46 us, 5.6 TB/s.
//
// GROUPED products have the rows of a block of experts: 16384 rows by 2 of 16 experts of 2048 x 4096 at 1300 to 1500
// TFLOP/s of useful work (tiles of 256 rows for experts of about 1000 leave an eighth to padding); 1554 rows
// of 24 experts of 1000 x 1366 read their weights at 3.4 to 4 TB/s, of 2048 x 4096 at 5.3.
#include "ffn_tc.cuh"

namespace im2win {
namespace ffn {
namespace {

template <int CG, int BN>
struct Tile {
    static constexpr int M = ROWS * CG;
    static constexpr int B_ROWS = BN / CG;  // rows of B a CTA stages
    static constexpr int A_BYTES = ROWS * BK * 2, B_BYTES = B_ROWS * BK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = STAGE <= 24 * 1024 ? 8 : 6;
    static constexpr int SMEM = STAGE * STAGES + 1024;  // + alignment
    // staged outputs besides, where they are needed (with them L1 has 28 KB instead of 60, and
    // the epilogue that reads kept values takes 39 us instead of 34)
    static constexpr int SMEM_STAGED = SMEM + EPI_WARPS * STAGED_WORDS * 4;
};

struct TcParams {
    CUtensorMap a[2], b[2];
    int M, N, KB;              // KB: blocks of 64 K steps of one segment
    int segs;                  // 2: the K blocks of a[1], b[1] follow those of a[0], b[0]
    int batch;                 // 2: a second product a[1], b[1] -> out2 of the same shape
    int tiles_m, tiles_n, tiles;
    int a_rows;                // rows of A's copies (fewer than ROWS when M is)
    int a_blocks, b_blocks;    // K outermost, whole blocks of 64 output indexes: one copy takes all of a stage's
    int bf16, act;
    void *out, *out2;
    unsigned char *kept;
    int64_t ldo;
    int vec;                   // bytes of output stores: 32, 16, or 2
    float *part;               // streamed: partial tiles
    int64_t part_ld, part_step;  // row pitch and distance between contributions, in floats
    int first;                 // the call's first launch: clears the status
    uint32_t *status;
    Groups groups;
    const float *scale;
    int table_at, rows_bound;  // where the groups lie in shared memory; rows of the grouped buffers
};

// Eight kept values: their upper halves and the bytes after them.
__device__ __forceinline__ void keep8(const F2 *v, uint4 &hi, uint2 &lo) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x, y;
        split(v[i], x, y);
        b[2 * i] = __float_as_uint(x), b[2 * i + 1] = __float_as_uint(y);
    }
    hi = make_uint4(__byte_perm(b[0], b[1], 0x7632), __byte_perm(b[2], b[3], 0x7632), __byte_perm(b[4], b[5], 0x7632),
                    __byte_perm(b[6], b[7], 0x7632));
    lo.x = __byte_perm(__byte_perm(b[0], b[1], 0x0051), __byte_perm(b[2], b[3], 0x0051), 0x5410);
    lo.y = __byte_perm(__byte_perm(b[4], b[5], 0x0051), __byte_perm(b[6], b[7], 0x0051), 0x5410);
}
// (The last eight bits, which were not kept, repeat the eight before them.)
__device__ __forceinline__ void kept8(F2 *v, const uint4 &hi, uint32_t lo0, uint32_t lo1) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = i < 2 ? lo0 : lo1;
        const uint32_t x = __byte_perm(h[i], lo, i & 1 ? 0x1066 : 0x1044), y = __byte_perm(h[i], lo, i & 1 ? 0x3277 : 0x3255);
        v[i] = f2(__uint_as_float(x), __uint_as_float(y));
    }
}
// 8 columns of a and b of a row, at kept_block().
__device__ __forceinline__ void keep_columns(unsigned char *at, const F2 *a, const F2 *b) {
    uint4 ha, hb;
    uint2 la, lb;
    keep8(a, ha, la);
    keep8(b, hb, lb);
    *reinterpret_cast<uint4 *>(at) = ha;
    *reinterpret_cast<uint4 *>(at + 512) = hb;
    *reinterpret_cast<uint4 *>(at + 1024) = make_uint4(la.x, la.y, lb.x, lb.y);
}

// The kept values of a chunk of row m: three vectors of each 8 columns.
struct KeptChunk {
    uint4 v[2][3];
};
__device__ __forceinline__ void fetch_kept(const TcParams &p, KeptChunk &k, int m, int m_end, int n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (m >= m_end || n + 8 * i >= p.N) continue;
        const unsigned char *at = p.kept + kept_block(m, n + 8 * i, p.N);
#pragma unroll
        for (int j = 0; j < 3; ++j) k.v[i][j] = *reinterpret_cast<const uint4 *>(at + 512 * j);
    }
}

// Outputs of a chunk of rows m0 + lane from their accumulator values v (and u, or kept), columns
// from n; every lane of the warp is here. Rows end at m_end. WIDE: outputs in fp32. scale: the row's.
template <int EPI, bool WIDE>
__device__ __forceinline__ void finish_chunk(const TcParams &p, F2 (&v)[PAIRS], F2 (&u)[PAIRS], const KeptChunk &k, int m0,
                                             int n, int m_end, uint16_t *out, uint32_t *stage, float scale) {
    const int m = m0 + (threadIdx.x & 31);
    if (n >= p.N) return;
    const int64_t at = (int64_t)m * p.ldo + n;
    if (WIDE) {
        ulonglong2 *to = reinterpret_cast<ulonglong2 *>(static_cast<float *>(p.out) + at);
        if (m >= m_end) return;
#pragma unroll
        for (int i = 0; i < PAIRS / 2; ++i)
            if (4 * i < p.ldo - n) to[i] = make_ulonglong2(v[2 * i].v, v[2 * i + 1].v);
        return;
    }
    if (EPI == EPI_STORE) {
        if (p.vec == 2) store_rows_staged(out + (int64_t)m0 * p.ldo + n, p.ldo, v, min(32, m_end - m0), p.N - n, p.bf16, stage);
        else if (m < m_end) store_row(out + at, v, p.N - n, p.vec, p.bf16);
        return;
    }
    if (m >= m_end) return;
    const int left = (int)(p.ldo - n);  // own buffers: whole vectors, whose last may pass N
    if (EPI == EPI_GATED) {
        F2 a[PAIRS];
        if (p.kept) {
            gate_values<PAIRS, true>(p.act, v, u, a);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (8 * i < left) keep_columns(p.kept + kept_block(m, n + 8 * i, p.N), a + 4 * i, u + 4 * i);
            if (p.scale) {
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) a[i] = mul2(v[i], f2(scale));
                store_row(static_cast<uint16_t *>(p.out2) + at, a, left, p.vec, p.bf16);
            }
        } else {
            gate_values<PAIRS, false>(p.act, v, u, a);
        }
    } else {
        F2 du[PAIRS];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            F2 a[4], b[4];
            kept8(a, k.v[i][0], k.v[i][2].x, k.v[i][2].y);
            kept8(b, k.v[i][1], k.v[i][2].z, k.v[i][2].w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                du[4 * i + j] = mul2(v[4 * i + j], a[j]);
                v[4 * i + j] = mul2(v[4 * i + j], b[j]);
            }
        }
        store_row(static_cast<uint16_t *>(p.out2) + at, du, left, p.vec, p.bf16);
    }
    store_row(out + at, v, left, p.vec, p.bf16);
}

// GROUPED: rows of A by expert, each with its matrix of B (AK); or sums by expert of the rows (!AK).
template <int CG, int BN, bool AK, bool BKM, int EPI, bool GROUPED>
__global__ void __launch_bounds__(THREADS, 1) tc_product(const __grid_constant__ TcParams p) {
    using T = Tile<CG, BN>;
    extern __shared__ unsigned char dyn[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ alignas(8) uint64_t bars[2 * T::STAGES + 4];
    const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * T::STAGES;
    const uint32_t acc_full = empty + 8 * T::STAGES, acc_empty = acc_full + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int unit = blockIdx.x / CG, units = gridDim.x / CG;
    const Ctl ctl{&abort_flag, p.status};

    if (threadIdx.x >= 64 && threadIdx.x < 68) {  // the maps' first use is a microsecond away
        const int i = threadIdx.x & 1;
        const bool b = threadIdx.x >= 66;
        if (i == 0 || p.segs == 2 || p.batch == 2 || (b && EPI == EPI_GATED))
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(b ? &p.b[i] : &p.a[i])) : "memory");
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < T::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, CG * EPI_WARPS);
        }
        fence_mbar_init();
    }
    // Tensor memory before the wait for the launch before, but for a call's first launch: what ran
    // before that may still hold some on this SM, and wait for an SM itself.
    auto setup = [&] {
        if (warp == 2) alloc_tmem<CG>(smem_u32(&tmem_slot), 2 * BN);
        tc_fence_before();
        __syncthreads();
        if (CG == 2) cluster_sync();
        tc_fence_after();
    };
    if (!p.first) setup();
    allow_dependents();
    grid_dependency_wait();
    if (p.first) setup();
    const uint32_t tmem = tmem_slot;
    // (a wait of this launch gives up two seconds from now at the earliest, after this store)
    if (p.first && blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;
    const GroupTable table = group_table(dyn + p.table_at, p.groups.E);
    if (GROUPED) {
        if (warp == 3) fill_group_table<!AK>(table, p, T::M, lane);
        __syncthreads();
    }
    auto begin_walk = [&] {
        if constexpr (GROUPED) return GroupWalk<!AK>(p, table, T::M, unit, units);
        else return Walk(p, unit, units);
    };

    if (warp == 0 && lane == 0) {
        // ---- copies
        auto walk = begin_walk();
        Work w;
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        constexpr int b_box = EPI == EPI_GATED && CG == 1 ? BN / 2 : T::B_ROWS;
        const uint32_t a_bytes = AK ? p.a_rows * BK * 2 : (p.a_rows + 63) / 64 * 64 * BK * 2;
        uint32_t bytes = CG * (a_bytes + T::B_BYTES);
        while (ok && walk.next(w)) {
            const int m0 = w.tm * T::M + (int)rank * ROWS + (GROUPED && AK ? w.row0 : 0);
            // grouped rows: copies of 64, as many as the expert's rows (and their padding) take of the tile
            const int a_copies = GROUPED && AK ? min(max((w.pad_end - m0) / 64, 0), 2) : 0;
            if (GROUPED && AK) {
                const int all = CG == 2 ? min(max((w.pad_end - w.tm * T::M - w.row0) / 64, 0), 4) : a_copies;
                bytes = CG * T::B_BYTES + all * 64 * BK * 2;
            }
            for (int kb = w.k0; kb < w.k1; ++kb) {
                if (!(ok = bar_wait(empty + 8 * s, phase ^ 1, ctl, SITE_STAGE_EMPTY))) break;
                const uint32_t sa = base + s * T::STAGE, sb = sa + T::A_BYTES;
                const uint32_t bar = CG == 2 ? map_rank(full + 8 * s, 0) : full + 8 * s;
                if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
                const int seg = kb >= p.KB ? 1 : 0, k = (kb - seg * p.KB) * BK + (GROUPED && !AK ? w.row0 : 0);
                const CUtensorMap *ma = &p.a[seg | w.z], *mb = &p.b[seg | w.z];
                if (GROUPED && AK) {
                    for (int i = 0; i < a_copies; ++i) tma_2d<CG>(sa + i * 64 * BK * 2, ma, k, m0 + i * 64, bar);
                } else if (AK) {
                    tma_2d<CG>(sa, ma, k, m0, bar);
                } else if (p.a_blocks) {
                    tma_3d<CG>(sa, ma, 0, k, m0 / 64, bar);
                } else {
                    for (int i = 0; i < p.a_rows; i += 64) tma_2d<CG>(sa + i * BK * 2, ma, m0 + i, k, bar);
                }
                if (EPI == EPI_GATED) {  // gate rows, then up rows of the same hidden channels
                    const int n0 = w.tn * (BN / 2);
                    if (GROUPED) {
                        tma_3d<CG>(sb, &p.b[CG == 2 ? rank : 0], k, n0, w.e, bar);
                        if (CG == 1) tma_3d<CG>(sb + b_box * BK * 2, &p.b[1], k, n0, w.e, bar);
                    } else if (CG == 2) {
                        tma_2d<CG>(sb, &p.b[rank], k, n0, bar);
                    } else {
                        tma_2d<CG>(sb, &p.b[0], k, n0, bar);
                        tma_2d<CG>(sb + b_box * BK * 2, &p.b[1], k, n0, bar);
                    }
                } else {
                    const int n0 = w.tn * BN + (int)rank * T::B_ROWS;
                    if (GROUPED && AK) {
                        if (BKM) {
                            tma_3d<CG>(sb, mb, k, n0, w.e, bar);
                        } else if (p.b_blocks) {
                            tma_4d<CG>(sb, mb, 0, k, n0 / 64, w.e, bar);
                        } else {
#pragma unroll
                            for (int i = 0; i < T::B_ROWS; i += 64) tma_3d<CG>(sb + i * BK * 2, mb, n0 + i, k, w.e, bar);
                        }
                    } else if (BKM) {
                        tma_2d<CG>(sb, mb, k, n0, bar);
                    } else if (p.b_blocks) {
                        tma_3d<CG>(sb, mb, 0, k, n0 / 64, bar);
                    } else {
#pragma unroll
                        for (int i = 0; i < T::B_ROWS; i += 64) tma_2d<CG>(sb + i * BK * 2, mb, n0 + i, k, bar);
                    }
                }
                if (++s == T::STAGES) s = 0, phase ^= 1;
            }
        }
        if (ok) ok = drain(empty, T::STAGES, s, phase, ctl, SITE_STAGE_EMPTY);
        if (!ok) let_end();
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- MMAs
        auto walk = begin_walk();
        Work w;
        int s = 0, n_tile = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t idesc = make_idesc(p.bf16 != 0, T::M, BN) | (AK ? 0u : 1u << 15) | (BKM ? 0u : 1u << 16);
        // K-major: 8-row groups 1024 bytes apart, a K step of 16 is 32 bytes further in the
        // swizzled row. Else: blocks of 64 output indexes BK * 128 bytes apart, groups of 8
        // K rows 1024 bytes apart, a K step is two groups.
        const uint64_t da = smem_desc(base, AK ? 16u : BK * 128u, 1024u) | (2ull << 61);
        const uint64_t db = smem_desc(base + T::A_BYTES, BKM ? 16u : BK * 128u, 1024u) | (2ull << 61);
        constexpr uint32_t step_a = (AK ? 32u : 2048u) >> 4, step_b = (BKM ? 32u : 2048u) >> 4;
        while (ok && walk.next(w)) {
            const int buf = n_tile & 1;
            if (!(ok = bar_wait(acc_empty + 8 * buf, ((n_tile >> 1) & 1) ^ 1, ctl, SITE_ACC_EMPTY))) break;
            tc_fence_after();
            const uint32_t d = tmem + buf * BN;
            for (int kb = w.k0; kb < w.k1; ++kb) {
                if (!(ok = bar_wait(full + 8 * s, phase, ctl, SITE_STAGE_FULL))) break;
                tc_fence_after();
                const uint64_t off = (uint64_t)(s * T::STAGE) >> 4;
#pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                    mma<CG>(d, da + off + k * step_a, db + off + k * step_b, idesc, kb > w.k0 || k > 0);
                commit<CG>(empty + 8 * s);
                if (++s == T::STAGES) s = 0, phase ^= 1;
            }
            if (ok) commit<CG>(acc_full + 8 * buf);
            ++n_tile;
        }
        if (!ok) let_end();
    } else if (warp >= 4) {
        // ---- outputs: a warp for 32 rows and a share of the columns
        auto walk = begin_walk();
        Work w;
        int n_tile = 0;
        const int q = warp & 3, share = (warp - 4) >> 2;
        constexpr int SHARES = EPI_WARPS / 4;
        constexpr int COLS = EPI == EPI_GATED ? BN / 2 : BN;  // output columns of a tile
        const uint32_t empty_bar0 = CG == 2 ? map_rank(acc_empty, 0) : acc_empty;
        uint32_t *stage = reinterpret_cast<uint32_t *>(dyn + T::STAGES * T::STAGE + 1024) + (warp - 4) * STAGED_WORDS;
        while (walk.next(w)) {
            const int buf = n_tile & 1;
            const int m = w.tm * T::M + (int)rank * ROWS + q * 32 + lane + (GROUPED && AK ? w.row0 : 0);
            // (the padding of rows that will be summed over is stored too)
            const int m_end = !GROUPED || !AK ? p.M : EPI == EPI_STORE ? w.row_end : w.pad_end;
            constexpr int SPAN = COLS / SHARES;  // output columns of the warp
            // what was kept of a chunk is on its way before the chunk's sums are looked at
            KeptChunk kept;
            if (EPI == EPI_DGATED && (GROUPED ? w.whole : !p.part)) fetch_kept(p, kept, m, m_end, w.tn * COLS + share * SPAN);
            if (!warp_bar_wait(acc_full + 8 * buf, (n_tile >> 1) & 1, ctl, SITE_ACC_FULL)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + buf * BN + ((uint32_t)(q * 32) << 16);
            // Once the warp's last accumulator column is in registers the MMAs may have the
            // buffer; the arrival orders no memory but the loads, which are done, so it need not
            // wait for the stores under way.
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_relaxed(empty_bar0 + 8 * buf);
            };
            if (GROUPED ? p.part && !w.whole : p.part != nullptr) {
                constexpr int PART_SPAN = BN / SHARES;
                float *dst = GROUPED ? p.part + (int64_t)(2 * unit + w.slot) * T::M * BN + part_index((int)rank * ROWS + q * 32 + lane, 0, BN)
                                     : p.part + w.slot * p.part_step + ((int64_t)w.z * p.M + m) * p.part_ld + (int64_t)w.tn * BN;
#pragma unroll 1
                for (int c = share * PART_SPAN; c < (share + 1) * PART_SPAN; c += CHUNK) {
                    uint32_t r[CHUNK];
                    load_chunk(taddr + c, r);
                    tmem_wait_ld();
                    if (c + CHUNK == (share + 1) * PART_SPAN) release();
                    if (m < m_end) {
#pragma unroll
                        for (int i = 0; i < CHUNK / 4; ++i)
                            reinterpret_cast<uint4 *>(GROUPED ? dst + c * 32 : dst + c)[GROUPED ? 32 * i : i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                    }
                }
            } else {
                uint16_t *out = static_cast<uint16_t *>(w.z ? p.out2 : p.out);
                if (GROUPED && !AK) out += (int64_t)w.e * p.M * p.ldo;
                // nothing accumulates where an expert has no rows, and the padding's outputs are zero
                // whatever the weights hold
                const float scale = GROUPED && EPI != EPI_STORE && p.scale && m < w.row_end ? p.scale[m] : 0.0f;
                const bool none = GROUPED && (AK ? EPI != EPI_STORE && m >= w.row_end : w.k1 == 0);
#pragma unroll 1
                for (int c = share * SPAN; c < (share + 1) * SPAN; c += CHUNK) {
                    uint32_t r[CHUNK], ru[CHUNK];
                    load_chunk(taddr + c, r);
                    if (EPI == EPI_GATED) load_chunk(taddr + BN / 2 + c, ru);
                    tmem_wait_ld();
                    if (c + CHUNK == (share + 1) * SPAN) release();
                    F2 v[PAIRS], u[PAIRS];
                    pairs_of(r, v);
                    if (EPI == EPI_GATED) pairs_of(ru, u);
                    if (GROUPED && none) {
#pragma unroll
                        for (int i = 0; i < PAIRS; ++i) v[i] = u[i] = f2(0.0f);
                    }
                    KeptChunk now = kept;
                    if (GROUPED && none && EPI == EPI_DGATED) now = KeptChunk{};
                    if (EPI == EPI_DGATED && c + CHUNK < (share + 1) * SPAN) fetch_kept(p, kept, m, m_end, w.tn * COLS + c + CHUNK);
                    if (GROUPED && EPI == EPI_DGATED) {
#pragma unroll
                        for (int i = 0; i < PAIRS; ++i) v[i] = mul2(v[i], f2(scale));
                    }
                    finish_chunk<EPI, GROUPED && AK && EPI == EPI_STORE>(p, v, u, now, m - lane, w.tn * COLS + c, m_end, out,
                                                                         stage, scale);
                }
            }
            ++n_tile;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();  // (a release: the other CTA's arrivals here have been made)
    tc_fence_after();
    if (warp == 2) free_tmem<CG>(tmem, 2 * BN);
}

// Eight output columns of row m from their sums v (GATED: g, and u); none: whatever was kept, they are zero.
template <int EPI>
__device__ __forceinline__ void finish_octet(const TcParams &p, F2 (&v)[4], F2 (&u)[4], int m, int n, void *out, float scale,
                                             bool none = false) {
    const int left = min(8, p.N - n);
    const int64_t at = (int64_t)m * p.ldo + n;
    auto put = [&](uint16_t *dst, const F2(&r)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            split(r[i], a, b);
            w[i] = pack2(a, b, p.bf16);
        }
        if (p.vec >= 16 && left == 8) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) dst[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        }
    };
    if (EPI == EPI_GATED) {
        F2 a[4];
        if (p.kept) {
            gate_values<4, true>(p.act, v, u, a);
            keep_columns(p.kept + kept_block(m, n, p.N), a, u);
            if (p.scale) {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = mul2(v[i], f2(scale));
                put(static_cast<uint16_t *>(p.out2) + at, a);
            }
        } else {
            gate_values<4, false>(p.act, v, u, a);
        }
    } else if (EPI == EPI_DGATED) {
        const uint4 *from = reinterpret_cast<const uint4 *>(p.kept + kept_block(m, n, p.N));
        const uint4 nothing = make_uint4(0, 0, 0, 0);
        const uint4 ha = none ? nothing : from[0], hb = none ? nothing : from[32], lo = none ? nothing : from[64];
        F2 a[4], b[4];
        kept8(a, ha, lo.x, lo.y);
        kept8(b, hb, lo.z, lo.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = mul2(v[i], a[i]);
            v[i] = mul2(v[i], b[i]);
        }
        put(static_cast<uint16_t *>(p.out2) + at, a);
    }
    put(static_cast<uint16_t *>(out) + at, v);
}

// Adds the partial tiles of a streamed launch and finishes the outputs: one
// thread for eight consecutive output columns.
template <int BN, int EPI>
__global__ void __launch_bounds__(256) tc_join(const __grid_constant__ TcParams p, int tile_m, int units) {
    allow_dependents();
    grid_dependency_wait();
    constexpr int COLS = EPI == EPI_GATED ? BN / 2 : BN;
    int z, m, n, count;
    const float *src;
    if (!join_source<COLS, BN>(p, tile_m, units, z, m, n, count, src)) return;
    F2 v[4], u[4];
    add_partials<EPI == EPI_GATED, BN>(src, p.part_step, count, v, u);
    finish_octet<EPI>(p, v, u, m, n, z ? p.out2 : p.out, 0.0f);
}

// The same for a streamed launch over experts.
template <int CG, int BN, bool AK, int EPI>
__global__ void __launch_bounds__(256) tc_group_join(const __grid_constant__ TcParams p, int units) {
    using T = Tile<CG, BN>;
    constexpr int COLS = EPI == EPI_GATED ? BN / 2 : BN;
    extern __shared__ unsigned char dyn[];
    allow_dependents();
    grid_dependency_wait();
    const GroupTable table = group_table(dyn, p.groups.E);
    if (threadIdx.x < 32) fill_group_table<!AK>(table, p, T::M, threadIdx.x);
    __syncthreads();
    if (!AK) zero_empty<uint16_t>(table, p.groups.E, p.out, p.batch == 2 ? p.out2 : nullptr, (int64_t)p.M * p.ldo);
    Work w;
    int unit, last;
    if (!group_join_source(GroupSpace<!AK>(p, table, T::M), units, w, unit, last)) return;
    const int m_end = !AK ? p.M : EPI == EPI_STORE ? w.row_end : w.pad_end;
    for (int id = blockIdx.x % JOIN_SHARES * 256 + threadIdx.x; id < T::M * COLS / 8; id += JOIN_SHARES * 256) {
        const int row = id % T::M, col = id / T::M * 8;
        const int m = w.tm * T::M + row + (AK ? w.row0 : 0), n = w.tn * COLS + col;
        if (m >= m_end || n >= p.N) continue;
        F2 v[4], u[4];
        add_parts<EPI == EPI_GATED>(p.part, T::M, BN, row, col, unit, last, v, u);
        if (AK && EPI == EPI_STORE) {
            ulonglong2 *to = reinterpret_cast<ulonglong2 *>(static_cast<float *>(p.out) + (int64_t)m * p.ldo + n);
            to[0] = make_ulonglong2(v[0].v, v[1].v), to[1] = make_ulonglong2(v[2].v, v[3].v);
            continue;
        }
        const bool none = AK && m >= w.row_end;
        const float scale = AK && p.scale && !none ? p.scale[m] : 0.0f;
        if (none || EPI == EPI_DGATED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = none ? f2(0.0f) : mul2(v[i], f2(scale)), u[i] = none ? f2(0.0f) : u[i];
        }
        void *out = w.z ? p.out2 : p.out;
        if (!AK) out = static_cast<uint16_t *>(out) + (int64_t)w.e * p.M * p.ldo;
        finish_octet<EPI>(p, v, u, m, n, out, scale, none);
    }
}

template <int CG, int BN, bool AK, bool BKM, int EPI, bool GROUPED>
cudaError_t launch_shape(TcParams &p, const TcPlan &pl, cudaStream_t st) {
    using T = Tile<CG, BN>;
    constexpr auto kernel = tc_product<CG, BN, AK, BKM, EPI, GROUPED>;
    // (a streamed launch over experts finishes whole tiles itself)
    p.table_at = EPI == EPI_STORE && p.vec == 2 && (GROUPED || !p.part) ? T::SMEM_STAGED : T::SMEM;
    const int smem = p.table_at + (GROUPED ? group_table_bytes(p.groups.E) : 0);
    cudaError_t e = allow_smem<kernel>(T::SMEM_STAGED + (GROUPED ? group_table_bytes(MAX_EXPERTS) : 0));
    if (e != cudaSuccess) return e;
    e = launch_with(kernel, pl.units * CG, THREADS, smem, CG, st, p);
    if (e != cudaSuccess || !p.part) return e;
    if constexpr (GROUPED) {
        return launch_with(tc_group_join<CG, BN, AK, EPI>, group_join_blocks(pl.units, !AK), 256, group_table_bytes(p.groups.E), 1, st, p, pl.units);
    } else {
        return launch_with(tc_join<BN, EPI>, join_blocks(p), 256, 0, 1, st, p, T::M, pl.units);
    }
}

template <int CG, int BN, bool GROUPED>
cudaError_t launch_tile(TcParams &p, const TcPlan &pl, const Product &d, cudaStream_t st) {
    if (d.epi == EPI_GATED) return launch_shape<CG, BN, true, true, EPI_GATED, GROUPED>(p, pl, st);
    if (d.epi == EPI_DGATED) return launch_shape<CG, BN, true, false, EPI_DGATED, GROUPED>(p, pl, st);
    if (!d.a0.k_major) return launch_shape<CG, BN, false, false, EPI_STORE, GROUPED>(p, pl, st);
    if (d.b0.k_major) return launch_shape<CG, BN, true, true, EPI_STORE, GROUPED>(p, pl, st);
    return launch_shape<CG, BN, true, false, EPI_STORE, GROUPED>(p, pl, st);
}

cudaError_t launch_narrow(TcParams &p, const TcPlan &pl, const Product &d, cudaStream_t st) {
    if (d.epi == EPI_GATED) return launch_shape<2, 128, true, true, EPI_GATED, true>(p, pl, st);
    if (d.epi == EPI_DGATED) return launch_shape<2, 128, true, false, EPI_DGATED, true>(p, pl, st);
    if (d.b0.k_major) return launch_shape<2, 128, true, true, EPI_STORE, true>(p, pl, st);
    return launch_shape<2, 128, true, false, EPI_STORE, true>(p, pl, st);
}

}  // namespace

TcPlan plan_tc(const Product &d) {
    // A K block takes the same time in either shape (the pair's MMAs, four times as many; the
    // single CTA's shared-memory fill), outputs a little over half of it on the smaller tile.
    const double epi = d.epi == EPI_DGATED ? 4 : d.epi == EPI_GATED ? (d.kept ? 3 : 2.1) : 1.8;
    if (d.groups.E) {
        TcPlan best = plan_groups(d, 2, 256, 0.345, epi);
        const TcPlan single = plan_groups(d, 1, 128, 0.335, 0.55 * epi + 0.1);
        if (single.cost < best.cost) best = single;
        // Narrower tiles where about one tile of rows reads an expert: the weights are most of what is copied, and
        // the waves come out more even. (With many tiles the rows are copied twice as often: 46 us instead of 40 us
        // for 25088 rows of 2 x 1024 by 256 columns.)
        const TcPlan narrow = plan_groups(d, 2, 128, 0.26, 0.55 * epi + 0.1);
        return d.a0.k_major && d.rows <= 256.0 * d.groups.E && narrow.cost < best.cost ? narrow : best;
    }
    const TcPlan pair = plan_tiles(d, 2, 256, 0.345, epi), single = plan_tiles(d, 1, 128, 0.335, 0.55 * epi + 0.1);
    return single.cost < pair.cost ? single : pair;
}

cudaError_t launch_tc(const Product &d, bool bf16, uint32_t *status, bool first, void *part, cudaStream_t st) {
    const TcPlan pl = plan_tc(d);
    TcParams p = {};
    p.M = d.M; p.N = d.N; p.KB = (d.K + BK - 1) / BK;
    const bool two = d.a1.p != nullptr;
    p.segs = d.epi != EPI_GATED && two && !d.batch ? 2 : 1;
    p.batch = d.batch ? 2 : 1;
    p.groups = d.groups;
    p.scale = d.scale;
    p.rows_bound = d.a0.k_major ? d.M : d.K;
    const int stack = d.a0.k_major ? d.groups.E : 0, matrices = d.groups.E && !d.a0.k_major ? d.groups.E : 1;
    p.tiles_m = pl.tiles_m; p.tiles_n = pl.tiles_n; p.tiles = matrices * p.batch * pl.tiles_m * pl.tiles_n;
    p.a_rows = std::min(ROWS, (d.M + 7) / 8 * 8);
    const int b_box = d.epi == EPI_GATED && pl.cg == 1 ? pl.bn / 2 : pl.bn / pl.cg;
    p.a_blocks = !d.a0.k_major && d.M % 64 == 0;
    p.b_blocks = !d.b0.k_major && d.N % 64 == 0;
    if (stack) p.a_rows = 64;  // (of one copy)
    if (!encode(p.a[0], d.a0, 0, d.M, d.K, p.a_rows, p.a_blocks) || !encode(p.b[0], d.b0, 0, d.N, d.K, b_box, p.b_blocks, stack))
        return cudaErrorInvalidValue;
    if (two && !encode(p.a[1], d.a1, 0, d.M, d.K, p.a_rows, p.a_blocks)) return cudaErrorInvalidValue;
    if (d.b1.p && !encode(p.b[1], d.b1, 0, d.N, d.K, b_box, p.b_blocks, stack)) return cudaErrorInvalidValue;
    p.bf16 = bf16; p.act = d.act;
    p.out = d.out; p.out2 = d.out2; p.kept = static_cast<unsigned char *>(d.kept); p.ldo = d.ldo;
    p.vec = d.ldo % 16 == 0 && aligned_to(d.out, 32) && aligned_to(d.out2, 32) ? 32 : d.ldo % 8 == 0 ? 16 : 2;
    if (pl.streamed) {
        p.part = static_cast<float *>(part);
        p.part_ld = pl.part_ld;
        p.part_step = pl.part_step;
    }
    p.status = status;
    p.first = first;
    if (d.groups.E) {
        if (pl.cg == 1) return launch_tile<1, 128, true>(p, pl, d, st);
        return pl.bn == 256 ? launch_tile<2, 256, true>(p, pl, d, st) : launch_narrow(p, pl, d, st);
    }
    return pl.cg == 2 ? launch_tile<2, 256, false>(p, pl, d, st) : launch_tile<1, 128, false>(p, pl, d, st);
}

}  // namespace ffn
}  // namespace im2win
