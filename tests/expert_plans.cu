// What tests/test_expert_plans.py asks the host code of the group norm and the experts' products
// about shapes; nothing here runs on a GPU.
#include "expert_ffn.cuh"
#include "group_norm.cuh"

extern "C" {

// Units of a grouped product (0: no plan), whether its K is dealt out, and the bytes of its partial tiles. summed: over the
// grouped rows; else they are the rows of the product. two: a second pair of operands, joined (1) or apart (2).
int group_product_units(int f32, int summed, int M, int N, int K, int E, int64_t pairs, int kind, int two, int *streamed,
                        int64_t *part) {
    im2win::ffn::Product p;
    const void *some = reinterpret_cast<const void *>(16);
    p.M = M, p.N = N, p.K = K, p.epi = kind, p.batch = two == 2;
    p.a0.p = p.b0.p = some;
    p.a0.k_major = !summed;
    if (two || kind == im2win::ffn::EPI_GATED) p.b1.p = some;
    if (two) p.a1.p = some;
    p.groups.E = E;
    p.rows = (double)pairs;
    const im2win::ffn::TcPlan pl = f32 ? im2win::ffn::plan_f32(p) : im2win::ffn::plan_tc(p);
    *streamed = pl.streamed;
    *part = (int64_t)pl.part_bytes;
    return pl.units;
}

int64_t expert_grouped_rows(int64_t pairs, int64_t E) { return im2win::ffn::grouped_rows(pairs, E); }

// The group norm's cut: out = resident, chunks, positions a chunk, channels a slab, bytes of the tiles, of all shared memory,
// vector, slabs; or, for one position an image, 2, blocks of rows, rows and lanes of a block, lanes of a group, 0, vector, slabs.
void group_norm_cut(int64_t N, int64_t P, int C, int G, int size, int maps, int64_t *out) {
    im2win::gnorm::GroupArgs a = {};
    a.N = N, a.P = P, a.C = C, a.G = G, a.D = C / G;
    if (im2win::gnorm::cut_rows(a, size)) {
        const int64_t r[] = {2, a.chunks, a.rows, a.cols, a.lanes, 0, im2win::gnorm::vector_of(a.D, size), a.slabs};
        for (int i = 0; i < 8; ++i) out[i] = r[i];
        return;
    }
    if (!im2win::gnorm::cut_resident(a, size, maps)) im2win::gnorm::cut(a, size, maps);
    const int v = im2win::gnorm::vector_of(C, size);
    const int64_t r[] = {a.resident, a.chunks, a.len, a.resident ? a.slab : a.cols * v, a.tile, a.smem, v, a.slabs};
    for (int i = 0; i < 8; ++i) out[i] = r[i];
}

}  // extern "C"
