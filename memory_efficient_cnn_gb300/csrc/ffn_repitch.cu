// Copies of dense matrices to rows of a whole number of 16-byte vectors, which the
// tensor-core products' copies need: 16-bit ones whose width is no multiple of 8,
// and fp32 ones as three bf16 planes.
#include "gated_ffn.cuh"
#include "tc_ptx.cuh"

namespace im2win {
namespace ffn {
namespace {

struct List {
    Repitch m[5];
    int64_t first[6];  // first vector of each matrix, then their total
    int count;
};

// One 16-byte output vector per thread from the widest loads that every row's start
// allows; elements past a row's end are written as zero.
__global__ void __launch_bounds__(256) repitch(const __grid_constant__ List l) {
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= l.first[l.count]) return;
    int i = 0;
    while (i + 1 < l.count && id >= l.first[i + 1]) ++i;
    const Repitch m = l.m[i];
    const int vecs = (m.cols + 7) / 8;
    const int64_t row = (id - l.first[i]) / vecs;
    const int c = (int)(id - l.first[i] - row * vecs) * 8;
    const uint16_t *src = static_cast<const uint16_t *>(m.src) + row * m.cols + c;
    uint32_t v[4];
    if (m.cols % 2 == 0) {  // rows start on 4 bytes
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = c + 2 * e < m.cols ? *reinterpret_cast<const uint32_t *>(src + 2 * e) : 0u;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t x = c + e < m.cols ? src[e] : 0u;
            v[e / 2] = e % 2 ? v[e / 2] | (x << 16) : x;
        }
    }
    reinterpret_cast<uint4 *>(m.dst)[row * vecs + c / 8] = make_uint4(v[0], v[1], v[2], v[3]);
}

// fp32: eight elements a thread, to each of the three planes.
__global__ void __launch_bounds__(256) split_planes(const __grid_constant__ List l) {
    tc::allow_dependents();
    tc::grid_dependency_wait();
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= l.first[l.count]) return;
    int i = 0;
    while (i + 1 < l.count && id >= l.first[i + 1]) ++i;
    const Repitch m = l.m[i];
    const int vecs = (m.cols + 7) / 8;
    const int64_t row = (id - l.first[i]) / vecs;
    const int c = (int)(id - l.first[i] - row * vecs) * 8;
    const float *src = static_cast<const float *>(m.src) + row * m.cols + c;
    uint32_t v[3][4];
    if (m.cols % 4 == 0 && c + 8 <= m.cols) {
        const float4 a = reinterpret_cast<const float4 *>(src)[0], b = reinterpret_cast<const float4 *>(src)[1];
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint16_t p[3];
            split_f32(x[e], p[0], p[1], p[2]);
#pragma unroll
            for (int q = 0; q < 3; ++q) v[q][e / 2] = e % 2 ? v[q][e / 2] | ((uint32_t)p[q] << 16) : p[q];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint16_t p[3];
            split_f32(c + e < m.cols ? src[e] : 0.0f, p[0], p[1], p[2]);
#pragma unroll
            for (int q = 0; q < 3; ++q) v[q][e / 2] = e % 2 ? v[q][e / 2] | ((uint32_t)p[q] << 16) : p[q];
        }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
        reinterpret_cast<uint4 *>(m.dst)[((int64_t)q * m.rows + row) * vecs + c / 8] =
            make_uint4(v[q][0], v[q][1], v[q][2], v[q][3]);
}

}  // namespace

cudaError_t launch_repitch(const Repitch *list, int count, bool f32, cudaStream_t st) {
    List l;
    l.count = count;
    l.first[0] = 0;
    for (int i = 0; i < count; ++i) {
        l.m[i] = list[i];
        l.first[i + 1] = l.first[i] + (int64_t)list[i].rows * ((list[i].cols + 7) / 8);
    }
    const int64_t blocks = (l.first[count] + 255) / 256;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (f32) split_planes<<<(unsigned)blocks, 256, 0, st>>>(l);
    else repitch<<<(unsigned)blocks, 256, 0, st>>>(l);
    return cudaGetLastError();
}

}  // namespace ffn
}  // namespace im2win
