// What the tensor-core products of the gated feed-forward share: PTX of CTA pairs,
// the walk over tiles and K blocks, operand tensor maps and launches.
#pragma once

#include <algorithm>
#include <cmath>

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
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int e, uint32_t bar) {
    if (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(e), "r"(bar)
            : "memory");
    else
        tma_load_4d(dst, map, x, y, z, e, bar);
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
    // Grouped rows of A: the tile's expert, its first row, and the ends of its rows without and
    // with the padding. Grouped sums: the expert, its first row, of which the K blocks count.
    int e, row0, row_end, pad_end;
    bool whole;  // grouped: the run is all of its tile
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

// The groups as the roles of a CTA read them, in shared memory: the experts' first rows, their counts, and
// where their work begins: of rows of A in tiles, of sums in K blocks of all tiles of a matrix.
struct GroupTable {
    int *begin, *count, *first;
};
__host__ __device__ inline int group_table_bytes(int E) { return (3 * E + 1) * 4; }
__device__ inline GroupTable group_table(void *smem, int E) {
    int *p = static_cast<int *>(smem);
    return {p, p + E, p + 2 * E};
}
// Filled by one warp. (A backward call gets the groups from a buffer of the caller's: whatever it
// holds, no row at or past rows_bound is touched.)
template <bool SUMMED, typename P>
__device__ inline void fill_group_table(const GroupTable &t, const P &p, int tile_m, int lane) {
    const Groups &g = p.groups;
    int before = 0;
    for (int e0 = 0; e0 < g.E; e0 += 32) {
        const int e = e0 + lane;
        const int begin = e < g.E ? min(max(g.begin[e], 0), p.rows_bound) / GROUP_ROWS * GROUP_ROWS : 0;
        const int count = e < g.E ? min(max(g.count[e], 0), p.rows_bound - begin) : 0;
        const int work = SUMMED ? (count + BK - 1) / BK * p.tiles_m * p.tiles_n : (count + tile_m - 1) / tile_m * p.tiles_n;
        int sum = work;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (e < g.E) t.begin[e] = begin, t.count[e] = count, t.first[e] = before + sum - work;
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) t.first[g.E] = before;
}

// The K blocks of a grouped launch in one order: tile after tile of an expert (in bands as above), expert
// after expert; SUMMED: first all of out, then all of out2.
template <bool SUMMED>
struct GroupSpace {
    GroupTable t;
    int KT, tiles_m, tiles_n, tile_m, E, batch;
    template <typename P>
    __device__ GroupSpace(const P &p, const GroupTable &table, int tile_m_)
        : t(table), KT(p.KB * p.segs), tiles_m(p.tiles_m), tiles_n(p.tiles_n), tile_m(tile_m_), E(p.groups.E), batch(p.batch) {}
    __device__ int64_t total() const { return (int64_t)t.first[E] * (SUMMED ? batch : KT); }
    // CTA groups that a streamed launch deals its blocks to: four blocks each at least
    __device__ int takers(int units) const { return (int)max((int64_t)1, min((int64_t)units, total() / 4)); }
    // the r-th tile of expert w.e
    __device__ void place(Work &w, int r) const {
        const int count = t.count[w.e], rows_m = SUMMED ? tiles_m : (count + tile_m - 1) / tile_m;
        w.row0 = t.begin[w.e];
        w.row_end = w.row0 + count;
        w.pad_end = w.row0 + (count + GROUP_ROWS - 1) / GROUP_ROWS * GROUP_ROWS;
        const int band = r / (8 * tiles_n), in = r - band * 8 * tiles_n;
        const int rows = min(8, rows_m - band * 8);
        w.tn = in / rows;
        w.tm = band * 8 + in - w.tn * rows;
    }
    __device__ int expert_of(int64_t at) const {  // first[e] <= at < first[e + 1]
        int e = 0, hi = E;
        while (hi - e > 1) {
            const int mid = (e + hi) / 2;
            if (t.first[mid] <= at) e = mid;
            else hi = mid;
        }
        return e;
    }
    // The tile with block `at` (below total()): w but for its K blocks; returns the block's place in it, of `len`.
    __device__ int locate(int64_t at, Work &w, int &len) const {
        int r, k;
        if (SUMMED) {
            w.z = at >= t.first[E] ? 1 : 0;
            const int in = (int)(at - (int64_t)w.z * t.first[E]);
            w.e = expert_of(in);
            len = (t.count[w.e] + BK - 1) / BK;
            r = (in - t.first[w.e]) / len;
            k = in - t.first[w.e] - r * len;
        } else {
            const int tile = (int)(at / KT);
            w.z = 0;
            w.e = expert_of(tile);
            len = KT;
            r = tile - t.first[w.e];
            k = (int)(at - (int64_t)tile * KT);
        }
        place(w, r);
        return k;
    }
};

// Walks a CTA group's work over experts: every units-th tile, or a share of the K blocks (streamed). A run
// that is part of its tile goes to the unit's first buffer of partial sums where it begins inside, and can
// only be the unit's first then, else to its second.
template <bool SUMMED>
struct GroupWalk {
    GroupSpace<SUMMED> space;
    int units;
    bool streamed;
    int64_t at, end;
    template <typename P>
    __device__ GroupWalk(const P &p, const GroupTable &table, int tile_m, int unit, int units_) : space(p, table, tile_m), units(units_) {
        streamed = p.part != nullptr;
        if (streamed) {
            const int64_t total = space.total();
            const int takers = space.takers(units);
            at = unit < takers ? stream_begin(total, takers, unit) : total;
            end = unit < takers ? stream_begin(total, takers, unit + 1) : total;
        } else {
            at = unit;
            end = SUMMED ? p.tiles : table.first[space.E];
        }
    }
    __device__ bool next(Work &w) {
        if (at >= end) return false;
        int len;
        if (streamed) {
            w.k0 = space.locate(at, w, len);
            w.k1 = (int)min((int64_t)len, w.k0 + end - at);
            w.slot = w.k0 == 0;
            w.whole = w.k0 == 0 && w.k1 == len;
            at += w.k1 - w.k0;
            return true;
        }
        w.k0 = w.slot = 0;
        w.whole = true;
        if (SUMMED) {  // (experts without rows too: their outputs are zero)
            const int per = space.tiles_m * space.tiles_n, m = (int)at / per;
            w.z = m / space.E;
            w.e = m - w.z * space.E;
            w.k1 = (space.t.count[w.e] + BK - 1) / BK;
            space.place(w, (int)at - m * per);
        } else {
            space.locate(at * space.KT, w, len);
            w.k1 = len;
        }
        at += units;
        return true;
    }
};

// ---- joining the partial tiles of a streamed grouped launch: JOIN_SHARES blocks for each border between
// two units. The tile that a border cuts is joined at its first border. (A block for every 256 octets of
// output columns took 13 us where these take 9.)
constexpr int JOIN_SHARES = 8;
inline int group_join_blocks(int units, bool summed) { return (units - 1) * JOIN_SHARES + (summed ? 64 : 0); }
// The block's tile w and the units whose parts it adds: `unit`'s second buffer, then the first ones of those up
// to `last`. False: nothing to do.
template <bool SUMMED>
__device__ __forceinline__ bool group_join_source(const GroupSpace<SUMMED> &space, int units, Work &w, int &unit, int &last) {
    const int i = blockIdx.x / JOIN_SHARES + 1;
    const int takers = space.takers(units);
    if (i >= takers || i >= units) return false;
    const int64_t total = space.total(), at = stream_begin(total, takers, i);
    int len;
    const int k = space.locate(at, w, len);
    const int64_t start = at - k;
    if (k == 0 || start < stream_begin(total, takers, i - 1)) return false;
    unit = i - 1, last = i;
    while (last + 1 < takers && stream_begin(total, takers, last + 1) < start + len) ++last;
    return true;
}
// Partial tiles lie in blocks of 32 rows by 4 columns, 16 bytes a row, so that the warp that writes 32 rows of one moves
// 512 contiguous bytes, and the one that reads them.
__device__ __forceinline__ int part_index(int row, int col, int bn) { return (row / 32 * (bn / 4) + col / 4) * 128 + row % 32 * 4; }
// Their sums (TWO: of g and u, half a tile's columns apart).
template <bool TWO>
__device__ __forceinline__ void add_parts(const float *part, int tile_m, int bn, int row, int col, int unit, int last, F2 (&v)[4],
                                          F2 (&u)[4]) {
    const int64_t tile = (int64_t)tile_m * bn;
    const float *from = part + part_index(row, col, bn);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = u[i] = f2(0.0f);
    auto add = [](F2(&sum)[4], const float *p) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 a = reinterpret_cast<const float4 *>(p)[32 * i];
            sum[2 * i] = add2(sum[2 * i], f2(a.x, a.y)), sum[2 * i + 1] = add2(sum[2 * i + 1], f2(a.z, a.w));
        }
    };
    for (int j = unit; j <= last; ++j) {
        const float *p = from + (2 * j + (j == unit ? 1 : 0)) * tile;
        add(v, p);
        if (TWO) add(u, p + bn / 8 * 128);
    }
}
// Zeros for the matrices of experts without rows, by the launch's last 64 blocks.
template <typename T>
__device__ __forceinline__ void zero_empty(const GroupTable &t, int E, void *out, void *out2, int64_t elements) {
    const int block = blockIdx.x - (gridDim.x - 64);
    if (block < 0) return;
    for (int e = 0; e < E; ++e) {
        if (t.count[e] > 0) continue;
        for (void *base : {out, out2}) {
            if (!base) continue;
            T *p = static_cast<T *>(base) + e * elements;
            if (elements * sizeof(T) % 16 == 0) {
                for (int64_t i = block * 256 + threadIdx.x; i < elements * (int64_t)sizeof(T) / 16; i += 64 * 256)
                    reinterpret_cast<uint4 *>(p)[i] = make_uint4(0, 0, 0, 0);
            } else {
                for (int64_t i = block * 256 + threadIdx.x; i < elements; i += 64 * 256) p[i] = T(0);
            }
        }
    }
}

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
// I is a number of whole blocks, (64, K, I / 64), which takes several in one copy. stack:
// so many such matrices behind one another, as the outermost axis (0: one, without it).
inline bool encode(CUtensorMap &map, const Operand &o, int plane, int I, int K, int rows, bool blocks, int stack = 0) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = map_encoder();
    if (!enc) return false;
    void *base = const_cast<uint16_t *>(static_cast<const uint16_t *>(o.p) + plane * o.plane);
    const cuuint64_t pitch = (cuuint64_t)o.ld * 2;
    cuuint64_t dims[4] = {(cuuint64_t)(o.k_major ? K : blocks ? 64 : I), (cuuint64_t)(o.k_major ? I : K),
                          (cuuint64_t)(blocks ? I / 64 : 1), 1};
    cuuint64_t strides[3] = {pitch, 128, 128};
    cuuint32_t box[4] = {64u, o.k_major ? (cuuint32_t)rows : (cuuint32_t)BK, (cuuint32_t)(rows / 64), 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    const cuuint32_t rank = blocks ? 3 : 2;
    if (stack) dims[rank] = (cuuint64_t)stack, strides[rank - 1] = pitch * (cuuint64_t)(o.k_major ? I : K), box[rank] = 1u;
    return enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT16, stack ? rank + 1 : rank, base, dims, strides, box, estr,
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

// The plan of a grouped product: tiles of 128 * cg rows and bn columns, whole or their K blocks dealt out
// evenly (streamed). The experts' shares are not known here; they are taken to be even, with the
// last tile of rows half full, and the largest expert to have 1.6 times its share of a sum. kb and epi as
// in plan_tiles; while few rows share an expert's weights, a K block takes no less than its part of
// reading them at 6 TB/s. Partial tiles, of which a unit has two at most, stay in L2.
inline TcPlan plan_groups(const Product &d, int cg, int bn, double kb, double epi) {
    const bool summed = !d.a0.k_major;
    const int tm = ROWS * cg, cols = d.epi == EPI_GATED ? bn / 2 : bn, z = d.batch ? 2 : 1, most = SMS / cg;
    TcPlan pl;
    pl.cg = cg, pl.bn = bn;
    pl.tiles_m = (d.M + tm - 1) / tm;
    pl.tiles_n = (d.N + cols - 1) / cols;
    const double E = std::min<double>(d.groups.E, d.rows);  // experts with rows
    double KT, tiles, largest, bound, read = 0;
    if (summed) {
        KT = d.rows / E / BK + 0.5;
        tiles = (double)z * E * pl.tiles_m * pl.tiles_n;
        read = KT * tiles * ((double)tm / pl.tiles_n + (double)bn / pl.tiles_m) * BK * 2 / 5e6;
        largest = 1.6 * KT;
        bound = (double)z * d.groups.E * pl.tiles_m * pl.tiles_n;
    } else {
        const double tiles_m = std::max(1.0, d.rows / E / tm + 0.5);  // of an expert
        KT = largest = (double)((d.K + BK - 1) / BK * (d.epi != EPI_GATED && d.a1.p ? 2 : 1));
        tiles = std::ceil(E * tiles_m) * pl.tiles_n;
        kb = std::max(kb, bn / tiles_m * BK * 2 * most / 6e6);
        // (every expert's last tile may hold one row)
        bound = std::min<double>((double)((int64_t)d.M / tm + d.groups.E), d.M) * pl.tiles_n;
    }
    pl.units = (int)std::min<double>(most, bound);
    const double waves = std::ceil(std::max(1.0, tiles / most));
    pl.cost = 4 + std::max(read, largest * kb + epi + (waves - 1) * std::max(KT * kb, epi));
    // Work counts stay in 32 bits. With more tiles streaming does not pay: whole tiles next to one another find
    // their operands in L2 (16384 rows by 2048 columns: 683 us streamed, 420 us plain; 45 tiles of 32 blocks on 152
    // CTAs in fp32: 30 us and 45 us).
    if (bound * (KT + 1) * 4 > 1e9 || tiles > most) return pl;
    const double part = (double)most * tm * bn * 4, blocks = tiles * KT;
    const double cost = 4 + std::max(std::max(read, std::max(4.0, blocks / most) * kb), tiles / most * epi) + epi + 4 + 1.5 * part / 10e6;
    if (cost >= pl.cost) return pl;
    pl.streamed = true;
    pl.cost = cost;
    pl.units = most;
    pl.part_bytes = (size_t)(2 * most) * tm * bn * 4;
    return pl;
}

}  // namespace
}  // namespace ffn
}  // namespace im2win
