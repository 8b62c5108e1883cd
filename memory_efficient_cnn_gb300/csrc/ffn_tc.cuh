// What the tensor-core products of the gated feed-forward share: PTX of CTA pairs,
// the walk over tiles and K blocks, operand tensor maps and launches.
#pragma once

#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gated_ffn.cuh"
#include "tc_ptx.cuh"

namespace im2win {
namespace ffn {
namespace {

using namespace im2win::tc;

constexpr int BK = 64;           // K steps of one stage: 128 bytes
constexpr int ROWS = 128;        // rows of A a CTA stages (its TMEM lanes)
constexpr int EPI_WARPS = 16;
constexpr int THREADS = 128 + 32 * EPI_WARPS;

// SMs the work is cut for. A constant, so that sizes and results depend on the
// shape alone.
constexpr int SMS = 152;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address in the cluster's shared memory of `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// An arrival that orders no memory: tensor memory that has been read (tcgen05.wait::ld and a
// fence before it) is handed back so. The barrier at the kernel's end releases it to the other
// CTA before that may exit.
__device__ __forceinline__ void arrive_relaxed(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
template <int CG>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    if (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    if (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
            : "memory");
    else
        mma_f16(d, a, b, idesc, accumulate);
}
// One arrival on `bar` of each CTA of the tile once the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (CG == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        mma_commit(bar);
}
template <int CG>
__device__ __forceinline__ void alloc_tmem(uint32_t slot, uint32_t cols) {
    if (CG == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(slot, cols);
        tmem_relinquish();
    }
}
template <int CG>
__device__ __forceinline__ void free_tmem(uint32_t addr, uint32_t cols) {
    if (CG == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        tmem_dealloc(addr, cols);
}

// One run of K blocks of one tile.
struct Work {
    int z, tm, tn;  // batch, tile row, tile column
    int k0, k1;     // K blocks, over all segments
    int slot;       // streamed: the run's place among the tile's
};

// The K blocks of a streamed launch are dealt to `units` CTA groups: unit i takes
// blocks [i * total / units, (i + 1) * total / units).
__host__ __device__ inline int64_t stream_begin(int64_t total, int units, int i) { return total * i / units; }
// The unit that holds block b: an estimate in fp32, off by one at most, and no
// 64-bit division (a joining thread spent microseconds on them). Unit i begins at
// or before b where total * i < (b + 1) * units.
__host__ __device__ inline int stream_unit(int64_t total, int units, int64_t b) {
    int i = (int)((float)b * ((float)units / (float)total));
    if (i > units - 1) i = units - 1;
    while (i + 1 < units && total * (i + 1) < (b + 1) * units) ++i;
    while (i > 0 && total * i >= (b + 1) * units) --i;
    return i;
}

// Walks a CTA group's work.
struct Walk {
    int KT, tiles, tiles_m, tiles_n, per_z, units, unit, streamed;
    int64_t at, end;  // streamed: K blocks; else: tiles
    template <typename P>
    __device__ Walk(const P &p, int unit_, int units_) {
        KT = p.KB * p.segs;
        tiles = p.tiles, tiles_m = p.tiles_m, tiles_n = p.tiles_n, per_z = tiles_m * tiles_n;
        units = units_, unit = unit_, streamed = p.part != nullptr;
        at = streamed ? stream_begin((int64_t)tiles * KT, units, unit) : unit;
        end = streamed ? stream_begin((int64_t)tiles * KT, units, unit + 1) : tiles;
    }
    __device__ bool next(Work &w) {
        if (at >= end) return false;
        int t;
        if (streamed) {
            t = (int)(at / KT);
            w.k0 = (int)(at - (int64_t)t * KT);
            w.k1 = (int)min((int64_t)KT, w.k0 + end - at);
            w.slot = unit - stream_unit((int64_t)tiles * KT, units, (int64_t)t * KT);
            at += w.k1 - w.k0;
        } else {
            t = (int)at;
            w.k0 = 0, w.k1 = KT, w.slot = 0;
            at += units;
        }
        w.z = t / per_z;
        t -= w.z * per_z;
        // bands of 8 tile rows, column by column, so that tiles in flight share operands in L2
        const int band = t / (8 * tiles_n), r = t - band * 8 * tiles_n;
        const int rows = min(8, tiles_m - band * 8);
        w.tn = r / rows;
        w.tm = band * 8 + r - w.tn * rows;
        return true;
    }
};

constexpr int CHUNK = 16;  // accumulator columns a warp turns into outputs at a time
constexpr int PAIRS = CHUNK / 2;

__device__ __forceinline__ void load_chunk(uint32_t taddr, uint32_t (&r)[CHUNK]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void pairs_of(const uint32_t (&r)[CHUNK], F2 (&v)[PAIRS]) {
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) v[i] = f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

constexpr int STAGED_WORDS = 32 * (PAIRS + 1);  // a warp's chunk of outputs

// A chunk of outputs of one row from fp32, rounded and packed.
__device__ __forceinline__ void pack_row(const F2 (&v)[PAIRS], uint32_t (&w)[PAIRS], int bf16) {
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        float lo, hi;
        split(v[i], lo, hi);
        w[i] = pack2(lo, hi, bf16);
    }
}
// Into a row of whole 16-byte vectors, `n` columns from here on (a multiple of 8).
__device__ __forceinline__ void store_row(uint16_t *dst, const F2 (&v)[PAIRS], int n, int vec, int bf16) {
    uint32_t w[PAIRS];
    pack_row(v, w, bf16);
    if (vec == 32 && n >= CHUNK) {  // a whole sector in one store
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        if (n >= CHUNK) reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
// A warp's chunk of 32 rows into rows of any pitch, through its part of shared memory, so
// that neighbouring lanes store neighbouring columns (a lane's own row in 2-byte stores took
// 78 us for 2 x 3326 x 914 outputs). rows, n: valid rows and columns.
__device__ __forceinline__ void store_rows_staged(uint16_t *dst, int64_t ldo, const F2 (&v)[PAIRS], int rows, int n, int bf16,
                                                  uint32_t *stage) {
    const int lane = threadIdx.x & 31;
    uint32_t w[PAIRS];
    pack_row(v, w, bf16);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) stage[lane * (PAIRS + 1) + i] = w[i];
    __syncwarp();
    if (ldo % 2 == 0) {  // 4-byte stores (rows and the first column are even)
#pragma unroll
        for (int it = 0; it < PAIRS; ++it) {
            const int row = it * 4 + lane / PAIRS, c = lane % PAIRS * 2;
            if (row < rows && c < n) *reinterpret_cast<uint32_t *>(dst + row * ldo + c) = stage[row * (PAIRS + 1) + c / 2];
        }
    } else {
        const uint16_t *half = reinterpret_cast<const uint16_t *>(stage);
#pragma unroll
        for (int it = 0; it < CHUNK; ++it) {
            const int row = it * 2 + lane / CHUNK, c = lane % CHUNK;
            if (row < rows && c < n) dst[row * ldo + c] = half[row * 2 * (PAIRS + 1) + c];
        }
    }
}

// g, u -> h = act(g) * u in g; N pairs. KEEP: act(g) and u act'(g) too, in a and u.
// The activation is chosen once for all values.
template <int N, bool KEEP>
__device__ __forceinline__ void gate_values(int act, F2 (&g)[N], F2 (&u)[N], F2 (&a)[N]) {
    with_act_device(act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (KEEP) {
                F2 d;
                act_both2<decltype(kind)::value>(g[i], a[i], d);
                g[i] = mul2(a[i], u[i]);
                u[i] = mul2(u[i], d);
            } else {
                g[i] = mul2(act_value2<decltype(kind)::value>(g[i]), u[i]);
            }
        }
    });
}

enum Site : uint32_t { SITE_STAGE_FULL = 32, SITE_STAGE_EMPTY, SITE_ACC_FULL, SITE_ACC_EMPTY };

// After a wait that gave up: copies and MMAs in flight end within microseconds; this
// gives them two milliseconds.
__device__ __forceinline__ void let_end() {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
}

// Waits until every slot of a ring of `slots` has been given back, the next one to be filled being
// `s` in `phase`. The arrivals that give slots back come by themselves, from MMAs that the other
// CTA of a pair may have issued: a CTA waits for all of them before it ends, so that none finds
// its shared memory gone.
__device__ __forceinline__ bool drain(uint32_t empty, int slots, int s, uint32_t phase, const Ctl &ctl, uint32_t site) {
    for (int i = 0; i < slots; ++i) {
        if (!bar_wait(empty + 8 * s, phase ^ 1, ctl, site)) return false;
        if (++s == slots) s = 0, phase ^= 1;
    }
    return true;
}

inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// An operand of I output indexes and K steps, copied `rows` output indexes at a
// time. K innermost: (K, I). Else: (I, K) in blocks of 64 output indexes, or, where
// I is a number of whole blocks, (64, K, I / 64), which takes several in one copy.
inline bool encode(CUtensorMap &map, const Operand &o, int plane, int I, int K, int rows, bool blocks) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc) return false;
    void *base = const_cast<uint16_t *>(static_cast<const uint16_t *>(o.p) + plane * o.plane);
    const cuuint64_t pitch = (cuuint64_t)o.ld * 2;
    const cuuint64_t dims[3] = {(cuuint64_t)(o.k_major ? K : blocks ? 64 : I), (cuuint64_t)(o.k_major ? I : K),
                                (cuuint64_t)(blocks ? I / 64 : 1)};
    const cuuint64_t strides[2] = {pitch, 128};
    const cuuint32_t box[3] = {64u, o.k_major ? (cuuint32_t)rows : (cuuint32_t)BK, (cuuint32_t)(rows / 64)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, blocks ? 3 : 2, base, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K, typename... A>
cudaError_t launch_with(K kernel, int grid, int block, size_t smem, int cluster, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- joining the partial tiles of a streamed launch, eight output columns a thread
template <typename P>
inline int join_blocks(const P &p) {
    const int64_t octets = (int64_t)p.batch * p.M * ((p.N + 7) / 8);
    return (int)((octets + 255) / 256);
}
// The thread's batch, row and first column, and its first partial sums: `count`
// contributions, p.part_step apart. COLS: output columns of a tile of BN.
template <int COLS, int BN, typename P>
__device__ __forceinline__ bool join_source(const P &p, int tile_m, int units, int &z, int &m, int &n, int &count,
                                            const float *&src) {
    // (few tiles: everything here fits 32 bits)
    const uint32_t octets = (uint32_t)(p.N + 7) / 8, id = blockIdx.x * 256u + threadIdx.x;
    const uint32_t zm = id / octets;
    z = zm >= (uint32_t)p.M ? 1 : 0;
    if (zm >= (uint32_t)p.batch * (uint32_t)p.M) return false;
    n = (int)(id - zm * octets) * 8, m = (int)zm - z * p.M;
    const int tm = m / tile_m, tn = n / COLS;
    // the tile's index in the order of Walk, and the units that hold its first and last block
    const int band = tm / 8, rows = min(8, p.tiles_m - band * 8);
    const int t = z * p.tiles_m * p.tiles_n + band * 8 * p.tiles_n + tn * rows + (tm - band * 8);
    const int KT = p.KB * p.segs;
    const int64_t total = (int64_t)p.tiles * KT;
    count = stream_unit(total, units, (int64_t)(t + 1) * KT - 1) - stream_unit(total, units, (int64_t)t * KT) + 1;
    src = p.part + (int64_t)zm * p.part_ld + (int64_t)tn * BN + (n - tn * COLS);
    return true;
}
// Their sums in the order of K (TWO: of g and u).
template <bool TWO, int BN>
__device__ __forceinline__ void add_partials(const float *src, int64_t step, int count, F2 (&v)[4], F2 (&u)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = u[i] = f2(0.0f);
    auto add = [](F2(&sum)[4], const float *from) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 a = reinterpret_cast<const float4 *>(from)[i];
            sum[2 * i] = add2(sum[2 * i], f2(a.x, a.y)), sum[2 * i + 1] = add2(sum[2 * i + 1], f2(a.z, a.w));
        }
    };
#pragma unroll 4
    for (int j = 0; j < count; ++j) {
        add(v, src + j * step);
        if (TWO) add(u, src + j * step + BN / 2);
    }
}

// The plan of a product on tiles of 128 * cg rows and bn columns: plain or streamed,
// whichever the estimate has faster. In microseconds, as measured over rows of 33
// to 12544 and blocks of 256 x 640 to 4096 x 10240: a launch takes 4 besides its
// work; a K block of one tile kb; a tile's outputs epi, which hides behind the next
// tile's K blocks; partial tiles are written and read at 6 TB/s and joined by a
// second launch of 4.
inline TcPlan plan_tiles(const Product &d, int cg, int bn, double kb, double epi) {
    const int KT = (d.K + BK - 1) / BK * (d.epi != EPI_GATED && d.a1.p && !d.batch ? 2 : 1);
    const int z = d.batch ? 2 : 1, tm = ROWS * cg, cols = d.epi == EPI_GATED ? bn / 2 : bn, most = SMS / cg;
    TcPlan pl;
    pl.cg = cg, pl.bn = bn;
    pl.tiles_m = (d.M + tm - 1) / tm;
    pl.tiles_n = (d.N + cols - 1) / cols;
    const int64_t tiles = (int64_t)z * pl.tiles_m * pl.tiles_n, total = tiles * KT;
    pl.units = (int)std::min<int64_t>(most, tiles);
    const int64_t waves = (tiles + pl.units - 1) / pl.units;
    pl.cost = 4 + KT * kb + epi + (double)(waves - 1) * std::max(KT * kb, epi);
    if (total > 0x3fffffffll) return pl;  // (streamed indexes stay in 32 bits)
    TcPlan st = pl;
    st.streamed = true;
    st.units = (int)std::min<int64_t>(most, std::max<int64_t>(1, total / 4));  // 4 blocks at least
    if (tiles > 8 * st.units || tiles % st.units == 0) return pl;  // (nearly) even without it
    // a tile meets at most this many runs of at least floor(total / units) blocks
    st.slots = (int)((KT - 1) / (total / st.units) + 2);
    st.part_ld = (int64_t)pl.tiles_n * bn;
    st.part_step = (int64_t)z * d.M * st.part_ld;
    st.part_bytes = (size_t)(st.slots * st.part_step) * 4;
    const double moved = (double)(tiles + st.units) * std::min(tm, d.M) * bn * 8;
    st.cost = 4 + (double)((total + st.units - 1) / st.units) * kb + bn / 128.0 + 4 + moved / 6e6;
    return st.cost < pl.cost ? st : pl;
}

}  // namespace
}  // namespace ffn
}  // namespace im2win
