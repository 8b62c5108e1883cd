// The whole forward pass of the gated feed-forward in one kernel, for few channels:
// h never leaves the SM.
//
// A pair of CTAs takes 256 rows of x, which stay in shared memory, and walks the
// hidden channels 64 at a time: g and u of a chunk are one product of 128 columns in
// tensor memory (the first CTA stages rows of w_gate, the second of w_up), eight warps
// make h of them and write it to shared memory as the next product's operand, and y +=
// h w_down^T accumulates beside them. Everything has two buffers, and even and odd
// chunks have eight warps each, so that one chunk's waits pass under the other's
// arithmetic; the two products are issued by a thread each, since g and u of the next
// chunk must not wait for h of this one (152 us with one thread, 110 us with two, at
// 200704 x 128 x 512 of gelu; 141 us in two kernels with h, 411 MB written and read,
// through memory). y of a tile is stored while the next one's first chunks are under way.
//
// What bounds it: the epilogue's instructions and waits, 1.24 us a chunk; the tensor
// cores are 28% busy.
#include "ffn_tc.cuh"

namespace im2win {
namespace ffn {
namespace {

constexpr int CHUNK_F = 64;                 // hidden channels of a chunk
constexpr int TILE_M = 2 * ROWS;
constexpr int X_BLOCK = ROWS * BK * 2, X_BYTES = 2 * 2 * X_BLOCK;  // x: two tiles of two blocks of 64 channels
constexpr int G_SLOTS = 8, G_BYTES = CHUNK_F * BK * 2;        // w_gate, w_up: slots of 64 rows by 64 channels
constexpr int D_SLOTS = 2, D_BYTES = 64 * CHUNK_F * 2;        // w_down: slots of up to 64 rows by a chunk
constexpr int H_BYTES = ROWS * CHUNK_F * 2;                   // h: two buffers
constexpr int SMEM = X_BYTES + G_SLOTS * G_BYTES + D_SLOTS * D_BYTES + 2 * H_BYTES + 1024;
constexpr int SMEM_STAGED = SMEM + EPI_WARPS * STAGED_WORDS * 4;
constexpr int BEHIND = 2;                   // chunks from g and u to y in the order of products (as many as buffers)
constexpr uint32_t Y_COLUMN = 2 * 2 * CHUNK_F, TMEM_COLUMNS = 512;  // (a power of two)

enum FusedSite : uint32_t {
    SITE_G_FULL = 48, SITE_G_EMPTY, SITE_D_FULL, SITE_D_EMPTY, SITE_X_FULL, SITE_X_EMPTY, SITE_GU_FULL, SITE_GU_EMPTY,
    SITE_H_FULL, SITE_H_EMPTY, SITE_Y_FULL, SITE_Y_EMPTY
};

struct FusedParams {
    CUtensorMap x, w[2], wd;
    int M, N, n_mma;     // rows, channels, columns of the product that makes them
    int KB, chunks, tiles;
    int bf16, act, vec;
    void *out;
    uint32_t *status;
};

// An arrival at the first CTA's barrier after which what this thread's warp wrote may be read there.
__device__ __forceinline__ void arrive_release(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Takes part in such arrivals, of a phase that has completed.
__device__ __forceinline__ void acquire_phase(uint32_t bar, uint32_t parity) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(bar), "r"(parity)
        : "memory");
}

// K-major, 128-byte-swizzled rows: 8-row groups 1024 bytes apart; a step of 16 is 32 bytes further.
__device__ __forceinline__ uint64_t operand_desc(uint32_t at) { return smem_desc(at, 16u, 1024u) | (2ull << 61); }

__global__ void __launch_bounds__(THREADS, 1) ffn_fused(const __grid_constant__ FusedParams p) {
    extern __shared__ unsigned char dyn[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ alignas(8) uint64_t bars[2 * (G_SLOTS + D_SLOTS + 2 + 2 + 2) + 2];
    const uint32_t x_at = (smem_u32(dyn) + 1023u) & ~1023u, g_at = x_at + X_BYTES, d_at = g_at + G_SLOTS * G_BYTES,
                   h_at = d_at + D_SLOTS * D_BYTES;
    uint32_t bar_at = smem_u32(bars);
    auto barriers = [&](int n) { const uint32_t at = bar_at; bar_at += 8 * n; return at; };
    const uint32_t g_full = barriers(G_SLOTS), g_empty = barriers(G_SLOTS), d_full = barriers(D_SLOTS),
                   d_empty = barriers(D_SLOTS), x_full = barriers(2), x_empty = barriers(2), gu_full = barriers(2),
                   gu_empty = barriers(2), h_full = barriers(2), h_empty = barriers(2), y_full = barriers(1),
                   y_empty = barriers(1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int unit = blockIdx.x / 2, units = gridDim.x / 2;
    const int my_tiles = (p.tiles - unit + units - 1) / units, total = my_tiles * p.chunks;
    const Ctl ctl{&abort_flag, p.status};

    if (threadIdx.x >= 64 && threadIdx.x < 68) {
        const CUtensorMap *maps[4] = {&p.x, &p.w[0], &p.w[1], &p.wd};
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[threadIdx.x - 64])) : "memory");
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2 * (G_SLOTS + D_SLOTS + 2 + 2 + 2) + 2; ++i) {
            const uint32_t bar = smem_u32(bars) + 8 * i;
            int count = 1;
            if (bar == gu_empty || bar == gu_empty + 8) count = EPI_WARPS;      // half of the warps of both CTAs
            if (bar == h_full || bar == h_full + 8) count = EPI_WARPS / 2 + (rank == 0);  // ... of this one, and the other's word
            if (bar == y_empty) count = 2 * EPI_WARPS;
            mbar_init(bar, count);
        }
        fence_mbar_init();
    }
    allow_dependents();
    grid_dependency_wait();
    // (after the wait: what ran before may hold tensor memory of this SM, and wait for an SM itself)
    if (warp == 2) alloc_tmem<2>(smem_u32(&tmem_slot), TMEM_COLUMNS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;

    if (warp == 0 && lane == 0) {
        // ---- copies, in the order in which the products take them
        int gs = 0, jd = 0;
        uint32_t g_phase = 0;
        bool ok = true;
        const uint32_t d_bytes = p.n_mma / 2 * CHUNK_F * 2;
        auto start = [&](uint32_t full, uint32_t bytes) {
            if (rank == 0) mbar_arrive_expect_tx(full, 2 * bytes);
            return map_rank(full, 0);
        };
        for (int i = 0, j = 0, tile = 0; ok && i < total + BEHIND; ++i) {
            if (i < total) {
                if (j == 0) {
                    const int s = tile & 1;
                    if (!(ok = bar_wait(x_empty + 8 * s, (tile >> 1 & 1) ^ 1, ctl, SITE_X_EMPTY))) break;
                    const uint32_t bar = start(x_full + 8 * s, p.KB * X_BLOCK);
                    const int m0 = (unit + tile * units) * TILE_M + (int)rank * ROWS;
                    for (int kb = 0; kb < p.KB; ++kb) tma_2d<2>(x_at + (s * 2 + kb) * X_BLOCK, &p.x, kb * BK, m0, bar);
                }
                for (int kb = 0; kb < p.KB; ++kb) {
                    if (!(ok = bar_wait(g_empty + 8 * gs, g_phase ^ 1, ctl, SITE_G_EMPTY))) break;
                    tma_2d<2>(g_at + gs * G_BYTES, &p.w[rank], kb * BK, j * CHUNK_F, start(g_full + 8 * gs, G_BYTES));
                    if (++gs == G_SLOTS) gs = 0, g_phase ^= 1;
                }
                if (!ok) break;
            }
            if (i >= BEHIND) {
                const int s = i & 1;
                if (!(ok = bar_wait(d_empty + 8 * s, ((i - BEHIND) >> 1 & 1) ^ 1, ctl, SITE_D_EMPTY))) break;
                tma_2d<2>(d_at + s * D_BYTES, &p.wd, jd * CHUNK_F, (int)rank * p.n_mma / 2, start(d_full + 8 * s, d_bytes));
                if (++jd == p.chunks) jd = 0;
            }
            if (++j == p.chunks) j = 0, ++tile;
        }
        // every arrival that is on its way to this CTA: buffer s of two has had `uses` / 2 rounds (h_empty, on
        // which this thread has not waited before, lags d_empty by less than a round: h was written after it)
        auto drain2 = [&](uint32_t bar, int uses, uint32_t site) {
            for (int s = 0; ok && s < 2; ++s) {
                const int rounds = (uses + 1 - s) / 2;
                if (rounds) ok = bar_wait(bar + 8 * s, (rounds - 1) & 1, ctl, site);
            }
        };
        if (ok) ok = drain(g_empty, G_SLOTS, gs, g_phase, ctl, SITE_G_EMPTY);
        drain2(x_empty, my_tiles, SITE_X_EMPTY);
        drain2(d_empty, total, SITE_D_EMPTY);
        drain2(h_empty, total, SITE_H_EMPTY);
        if (!ok) let_end();
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---- MMAs of g and u (a thread of their own: they must not wait for h of other chunks)
        int gs = 0;
        uint32_t g_phase = 0;
        bool ok = true;
        const uint32_t idesc = make_idesc(p.bf16 != 0, TILE_M, 2 * CHUNK_F);
        for (int i = 0, j = 0, tile = 0; ok && i < total; ++i) {
            const int buf = i & 1, xs = tile & 1;
            if (j == 0 && !(ok = bar_wait(x_full + 8 * xs, tile >> 1 & 1, ctl, SITE_X_FULL))) break;
            if (!(ok = bar_wait(gu_empty + 8 * buf, (i >> 1 & 1) ^ 1, ctl, SITE_GU_EMPTY))) break;
            for (int kb = 0; kb < p.KB; ++kb) {
                if (!(ok = bar_wait(g_full + 8 * gs, g_phase, ctl, SITE_G_FULL))) break;
                tc_fence_after();
                const uint64_t a = operand_desc(x_at + (xs * 2 + kb) * X_BLOCK), b = operand_desc(g_at + gs * G_BYTES);
#pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                    mma<2>(tmem + buf * 2 * CHUNK_F, a + 2 * k, b + 2 * k, idesc, kb > 0 || k > 0);
                commit<2>(g_empty + 8 * gs);
                if (++gs == G_SLOTS) gs = 0, g_phase ^= 1;
            }
            if (!ok) break;
            commit<2>(gu_full + 8 * buf);
            if (++j == p.chunks) j = 0, ++tile, commit<2>(x_empty + 8 * xs);
        }
        if (!ok) let_end();
    } else if (warp == 3 && lane == 0 && rank == 0) {
        // ---- MMAs of y
        bool ok = true;
        const uint32_t idesc = make_idesc(p.bf16 != 0, TILE_M, p.n_mma);
        for (int i = 0, j = 0, tile = 0; i < total; ++i) {
            const int s = i & 1;
            const uint32_t phase = i >> 1 & 1;
            if (!(ok = bar_wait(d_full + 8 * s, phase, ctl, SITE_D_FULL))) break;
            if (j == 0 && !(ok = bar_wait(y_empty, (tile & 1) ^ 1, ctl, SITE_Y_EMPTY))) break;
            if (!(ok = bar_wait(h_full + 8 * s, phase, ctl, SITE_H_FULL))) break;
            acquire_phase(h_full + 8 * s, phase);
            tc_fence_after();
            const uint64_t a = operand_desc(h_at + s * H_BYTES), b = operand_desc(d_at + s * D_BYTES);
#pragma unroll
            for (int k = 0; k < CHUNK_F / 16; ++k)
                mma<2>(tmem + Y_COLUMN, a + 2 * k, b + 2 * k, idesc, j > 0 || k > 0);
            commit<2>(d_empty + 8 * s);
            commit<2>(h_empty + 8 * s);
            if (++j == p.chunks) j = 0, ++tile, commit<2>(y_full);
        }
        if (!ok) let_end();
    } else if (warp == 1 && lane == 0) {
        // ---- the second CTA's h, to the thread that issues for both: a release to the cluster from
        // every warp of the epilogue took half a microsecond of each
        for (int i = 0; i < total; ++i) {
            if (!bar_wait(h_full + 8 * (i & 1), i >> 1 & 1, ctl, SITE_H_FULL)) break;
            arrive_release(map_rank(h_full + 8 * (i & 1), 0));
        }
    } else if (warp >= 4) {
        // ---- h: eight warps for even chunks and eight for odd ones, a warp for 32 rows and half
        // of the hidden channels. On its first chunk of a tile, once that is h, a warp stores its
        // share of y (every fourth 16 channels) of the tiles before.
        const int q = warp & 3, half = (warp - 4) >> 2 & 1, buf = (warp - 4) >> 3, row = q * 32 + lane;
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t gu_empty0 = map_rank(gu_empty + 8 * buf, 0), y_empty0 = map_rank(y_empty, 0);
        uint32_t *stage = reinterpret_cast<uint32_t *>(dyn + SMEM) + (warp - 4) * STAGED_WORDS;
        auto store_y = [&](int tile) {
            if (!warp_bar_wait(y_full, tile & 1, ctl, SITE_Y_FULL)) return false;
            tc_fence_after();
            const int m0 = (unit + tile * units) * TILE_M + (int)rank * ROWS + q * 32;
            uint16_t *out = static_cast<uint16_t *>(p.out) + (int64_t)m0 * p.N;
#pragma unroll 1
            for (int c = (half * 2 + buf) * CHUNK; c < p.n_mma; c += EPI_WARPS / 4 * CHUNK) {
                uint32_t r[CHUNK];
                load_chunk(taddr + Y_COLUMN + c, r);
                tmem_wait_ld();
                F2 v[PAIRS];
                pairs_of(r, v);
                const int rows = min(32, p.M - m0);
                if (p.vec == 2) {
                    if (c < p.N) store_rows_staged(out + c, p.N, v, rows, p.N - c, p.bf16, stage);
                } else if (c < p.N && lane < rows) {
                    store_row(out + (int64_t)lane * p.N + c, v, p.N - c, p.vec, p.bf16);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(y_empty0);
            return true;
        };
        // the 128-byte-swizzled layout that the copies give the other operands
        const uint32_t h_row = h_at + buf * H_BYTES + row / 8 * 1024 + row % 8 * 128;
        bool ok = true;
        int stored = 0, next = p.chunks;  // tiles whose y is stored; the first chunk that has one more before it
        for (int i = buf; ok && i < total; i += 2) {
            const uint32_t phase = i >> 1 & 1;
            if (!(ok = warp_bar_wait(gu_full + 8 * buf, phase, ctl, SITE_GU_FULL))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = half * 2 * CHUNK + c * CHUNK;
                uint32_t rg[CHUNK], ru[CHUNK], w[PAIRS];
                load_chunk(taddr + buf * 2 * CHUNK_F + col, rg);
                load_chunk(taddr + buf * 2 * CHUNK_F + CHUNK_F + col, ru);
                tmem_wait_ld();
                if (c == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_relaxed(gu_empty0);
                }
                F2 g[PAIRS], u[PAIRS], unused[PAIRS];
                pairs_of(rg, g);
                pairs_of(ru, u);
                gate_values<PAIRS, false>(p.act, g, u, unused);
                pack_row(g, w, p.bf16);
                if (c == 0) ok = warp_bar_wait(h_empty + 8 * buf, phase ^ 1, ctl, SITE_H_EMPTY);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(h_row + (((col / 8 + e) ^ (row % 8)) << 4)),
                                 "r"(w[4 * e]), "r"(w[4 * e + 1]), "r"(w[4 * e + 2]), "r"(w[4 * e + 3])
                                 : "memory");
            }
            if (!ok) break;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(h_full + 8 * buf);
            for (; ok && next <= i; next += p.chunks) ok = store_y(stored++);
        }
        while (ok && stored < my_tiles) ok = store_y(stored++);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // (a release: the other CTA's arrivals here have been made)
    tc_fence_after();
    if (warp == 2) free_tmem<2>(tmem, TMEM_COLUMNS);
}

}  // namespace

// Where the kernel covers the sizes: its estimated time, else zero. In microseconds, as
// measured: a chunk takes 1.1 with 64 channels and 1.24 with 128, the launch 5. (With
// more channels larger tiles do better, h through memory: 50176 x 256 x 1024 took 95
// us in a kernel like this, and takes 79 us in two products.)
double fused_cost(int64_t R, int64_t C, int64_t F) {
    if (C < 16 || C > 128 || F < CHUNK_F || R < TILE_M) return 0;
    const int64_t tiles = (R + TILE_M - 1) / TILE_M, chunks = (F + CHUNK_F - 1) / CHUNK_F;
    const int64_t waves = (tiles + SMS / 2 - 1) / (SMS / 2);
    if (waves * chunks > 0x3fffffff) return 0;
    return 5 + (double)(waves * chunks) * (0.96 + 0.0022 * (double)C);
}

cudaError_t launch_fused(const Fused &f, bool bf16, uint32_t *status, cudaStream_t st) {
    FusedParams p = {};
    p.M = f.R; p.N = f.C; p.n_mma = fused_columns(f.C);
    p.KB = (f.C + BK - 1) / BK;
    p.chunks = (f.F + CHUNK_F - 1) / CHUNK_F;
    p.tiles = (f.R + TILE_M - 1) / TILE_M;
    p.bf16 = bf16; p.act = f.act;
    p.out = f.y;
    p.vec = f.C % 16 == 0 && aligned_to(f.y, 32) ? 32 : f.C % 8 == 0 ? 16 : 2;
    p.status = status;
    if (!encode(p.x, f.x, 0, f.R, f.C, ROWS, false) || !encode(p.w[0], f.wg, 0, f.F, f.C, CHUNK_F, false) ||
        !encode(p.w[1], f.wu, 0, f.F, f.C, CHUNK_F, false) || !encode(p.wd, f.wd, 0, f.C, f.F, p.n_mma / 2, false))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(ffn_fused, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_STAGED);
    if (e != cudaSuccess) return e;
    return launch_with(ffn_fused, 2 * std::min(SMS / 2, p.tiles), THREADS, p.vec == 2 ? SMEM_STAGED : SMEM, 2, st, p);
}

}  // namespace ffn
}  // namespace im2win
