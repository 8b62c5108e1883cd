// Group norm over channels-last maps with its activation: the problem, how its
// sums over positions are cut, and the launchers (one translation unit for each type).
#pragma once

#include <algorithm>

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
};

constexpr int THREADS = 256;
constexpr int BATCH = 8;  // positions a thread has in flight

// Elements of a vector: 16 bytes where the channels allow, else pairs, else one.
inline int vector_of(int64_t C, int size) { return C % (16 / size) == 0 ? 16 / size : C % 2 == 0 ? 2 : 1; }

// Fills in the cut: eight blocks an SM, if the positions last. A constant number of SMs,
// so that results depend on the shape alone.
inline void cut(GroupArgs &a, int size) {
    const int vecs = a.C / vector_of(a.C, size);
    a.cols = std::min(vecs, THREADS);
    a.slabs = (vecs + a.cols - 1) / a.cols;
    a.rows = THREADS / a.cols;
    const int64_t most = (a.P + (int64_t)a.rows * BATCH - 1) / ((int64_t)a.rows * BATCH);
    const int64_t want = std::max<int64_t>(1, 152 * 8 / std::max<int64_t>(1, a.N * a.slabs));
    const int64_t chunks = std::max<int64_t>(1, std::min(most, want));
    a.len = std::max<int64_t>(1, (a.P + chunks - 1) / chunks);
    a.chunks = (int)std::max<int64_t>(1, (a.P + a.len - 1) / a.len);
}

template <typename T>
cudaError_t launch_forward(const GroupArgs &a, cudaStream_t st);
template <typename T>
cudaError_t launch_backward(const GroupArgs &a, cudaStream_t st);

}  // namespace gnorm
}  // namespace im2win
