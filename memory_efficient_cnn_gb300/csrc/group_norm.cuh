// Group norm over channels-last maps with its activation: the problem, how its
// sums over positions are cut, and the launchers (one translation unit for each type).
#pragma once

#include <algorithm>
#include <cmath>

#include "elem.cuh"

namespace im2win {
namespace gnorm {

// N images of P positions of C channels in G groups of D.
struct GroupArgs {
    const void *x, *dy, *w, *b;
    void *y, *dx, *dw, *db;
    float *stats;  // [N][G]: mean, 1 / deviation
    float *part;   // partial sums over chunks of positions, [2][N * chunks][C]
    float *sums;   // backward: [N][G][2], the means over a group that dx needs
    int64_t N, P;
    int C, G, D, act;
    float eps;
    // the cut: blocks of `cols` vectors (of `slabs` a position) by `rows` positions,
    // `chunks` of `len` positions an image
    int cols, slabs, rows, chunks;
    int64_t len;
    // resident: a cluster of `chunks` CTAs keeps the `slab` channels of an image on the chip
    bool resident;
    int slab, tile, smem;  // bytes: the tiles, and all
    int64_t part_rows;     // rows of the partial sums
    float *folded;         // backward: [2][folds][C], the partial sums of dw and db in `folds` runs of rows
    int folds;             // (0: they are few, and summed at once)
    int lanes;             // one position an image: lanes of a group (0: not so), `cols` of them a block and row
};

constexpr int THREADS = 256;
constexpr int64_t RESIDENT_BYTES = 16 << 20;
constexpr int MOST_SHARES = 8;  // CTAs of a cluster
constexpr size_t MAX_SMEM = 227 << 10;
constexpr int FEW = 4;  // positions a thread has at least, if there are as many

// Elements of a vector: 16 bytes where the channels allow, else pairs, else one.
inline int vector_of(int64_t C, int size) { return C % (16 / size) == 0 ? 16 / size : C % 2 == 0 ? 2 : 1; }

// The shared memory of a resident CTA besides its tile: a value for each element of a vector and
// thread (`sums` of them), their sums by channel and by group.
inline size_t resident_extra(int slab, int D, int vector, int sums) {
    return (size_t)sums * 4 * (THREADS * vector + std::max(THREADS, slab) + slab / D + 4);
}

// Whether an image's channels can stay on the chip between their sums and their outputs, and the
// cut if so: a slab of whole groups by all positions, over a cluster of up to eight CTAs, `maps`
// tensors of it (backward: x and dy). Slabs of 128 bytes of a position where they fit (shorter ones read
// parts of DRAM bursts), tiles of up to 48 KB, so that an SM has several CTAs in different phases;
// larger tiles only where the image does not fit otherwise.
inline bool cut_resident(GroupArgs &a, int size, int maps) {
    if (a.N * a.P * a.C * size * maps > RESIDENT_BYTES) return false;
    const int v = vector_of(a.C, size);
    int unit = a.D;
    while (unit % v) unit += a.D;
    for (const int64_t most : {48 << 10, 96 << 10, 190 << 10})
        for (const int bytes : {128, 64, 32}) {
            const int slab = std::min<int>(a.C, std::max(1, bytes / (unit * size)) * unit);
            if (slab / v > THREADS) return false;
            const int rows = THREADS / (slab / v);
            auto tile = [&](int s) {
                const int64_t len = (a.P + s - 1) / s;
                return (len + rows - 1) / rows * THREADS * v * size * maps;
            };
            int s = 1;
            while (s < MOST_SHARES && tile(s) > most) s *= 2;
            const size_t extra = resident_extra(slab, a.D, v, 2);
            if (tile(s) > most || tile(s) + extra > MAX_SMEM) continue;
            const int slabs = (a.C + slab - 1) / slab;
            // spread over the SMs while each thread has two positions
            while (s < MOST_SHARES && a.N * slabs * s < 304 && a.P >= (int64_t)rows * 4 * s) s *= 2;
            a.resident = true;
            a.slab = slab, a.slabs = slabs, a.chunks = s;
            a.len = (a.P + s - 1) / s;
            a.tile = (int)tile(s), a.smem = (int)(tile(s) + extra);
            return true;
        }
    return false;
}

// One position an image: a row's group belongs to up to 32 lanes with up to four vectors each. False where it is longer
// than that, or there are more positions.
inline bool cut_rows(GroupArgs &a, int size) {
    if (a.P != 1) return false;
    const int vecs = a.D / vector_of(a.D, size);
    int lanes = 1;
    while (lanes < 32 && lanes < vecs) lanes *= 2;
    if (vecs > 4 * lanes) return false;
    const int64_t slots = (int64_t)a.G * lanes;
    a.lanes = lanes;
    a.cols = (int)std::min<int64_t>(slots, THREADS);
    a.slabs = (int)((slots + a.cols - 1) / a.cols);
    a.rows = THREADS / a.cols;
    a.chunks = (int)std::max<int64_t>(1, std::min<int64_t>((a.N + a.rows - 1) / a.rows, 152 * 6 / a.slabs));
    a.part_rows = a.chunks;
    return true;
}

// Fills in the cut: as few chunks of positions as fill whole rounds of the blocks that the SMs hold at a time (four
// forward, three backward) to 93%, or else the best of up to four rounds. 64 images of 56 x 56 in 9 chunks are one
// round forward, where 14 left half of the second one empty.
inline void cut(GroupArgs &a, int size, int maps) {
    const int vecs = a.C / vector_of(a.C, size);
    a.cols = std::min(vecs, THREADS);
    a.slabs = (vecs + a.cols - 1) / a.cols;
    a.rows = THREADS / a.cols;
    const int64_t longest = std::max<int64_t>(1, (a.P + (int64_t)a.rows * FEW - 1) / ((int64_t)a.rows * FEW));
    const int64_t round = 152 * (maps == 1 ? 4 : 3), one = std::max<int64_t>(1, a.N * a.slabs);
    // (up to the first round they only fill it further)
    const int64_t first = std::max<int64_t>(1, std::min(longest, round * 93 / 100 / one));
    int64_t chunks = first;
    double best = 0;
    for (int64_t c = first; c <= longest && (c - 1) * one < 4 * round; ++c) {
        const int64_t blocks = c * one, rounds = (blocks + round - 1) / round;
        const double full = (double)blocks / (double)(rounds * round);
        if (full > best) best = full, chunks = c;
        if (best >= 0.93) break;
    }
    a.len = std::max<int64_t>(1, (a.P + chunks - 1) / chunks);
    a.chunks = (int)std::max<int64_t>(1, (a.P + a.len - 1) / a.len);
}

// Runs that the rows of partial sums of dw and db are summed in first. Up to 2048 rows a block of 32 channels adds up
// itself, 256 in a row; images of few positions can make millions, and then neither a run nor its block has more than
// about the square root of them (32768 x 4 x 32 in 16 bits: backward 1278 us without runs, 682 us with them; a million
// images of 2 x 8: 9e-4 and 1.4e-7 off in a sum of equal terms).
inline int folds_of(int64_t rows) { return rows <= 2048 ? 0 : (int)std::ceil(std::sqrt((double)rows)); }

template <typename T>
cudaError_t launch_forward(const GroupArgs &a, cudaStream_t st);
template <typename T>
cudaError_t launch_backward(const GroupArgs &a, cudaStream_t st);

}  // namespace gnorm
}  // namespace im2win
