// Host side of the paged decode: the split, the scratch layout and the launch.
#include "paged_decode.cuh"

namespace lssar {
namespace {

struct Layout {
    size_t stats, sums, o, counts, total;   // z first
};

Layout layout(const PagedDecode &pr, const paged::Split &sp) {
    const PagedCache &c = pr.c;
    const int keys = paged::tile_keys(c.d);
    const size_t rows = (size_t)c.B * sp.heads_rows, tiles = rows * ((c.capacity() + keys - 1) / keys);
    const size_t segments = (rows + (size_t)sp.ctas * paged::kChunksPerCta + 1) * sp.zg;
    auto r = [](size_t x) { return (x + 255) & ~(size_t)255; };
    Layout l;
    l.stats = is_reweight(pr.mode) || pr.scores ? r(tiles * sp.zg * keys * 4) : 0;
    l.sums = l.stats + (is_reweight(pr.mode) ? r(segments * 8) : 0);
    l.o = l.sums + r(segments * 8);
    l.counts = l.o + r(segments * c.d * 4);
    l.total = l.counts + (1 + 2 * rows) * 4;
    return l;
}

cudaError_t split(const PagedDecode &pr, paged::Split *sp) {
    const PagedCache &c = pr.c;
    const int G = pr.H / c.Hkv, keys = paged::tile_keys(c.d);
    sp->blocks = (G + paged::kHeads - 1) / paged::kHeads;
    sp->heads_rows = c.Hkv * sp->blocks;
    sp->zg = G < paged::kHeads ? G : paged::kHeads;
    const auto resident = c.half ? (c.d == 64 ? paged::fp16_d64_resident : paged::fp16_d128_resident)
                                 : (c.d == 64 ? paged::bf16_d64_resident : paged::bf16_d128_resident);
    const cudaError_t e = resident(pr.mode, &sp->ctas);
    const long long most = (long long)c.B * sp->heads_rows * ((c.capacity() + keys - 1) / keys);
    if (most < sp->ctas) sp->ctas = (int)most;
    if (sp->ctas > paged::kMaxCtas) sp->ctas = paged::kMaxCtas;
    sp->rows = c.B * sp->heads_rows;
    return e;
}

}  // namespace

cudaError_t paged_decode_workspace_bytes(const PagedDecode &pr, size_t *bytes) {
    paged::Split sp;
    const cudaError_t e = split(pr, &sp);
    if (e == cudaSuccess) *bytes = layout(pr, sp).total;
    return e;
}

cudaError_t launch_paged_decode(const PagedDecode &pr, void *ws, cudaStream_t stream) {
    paged::Args g;
    g.a = pr;
    cudaError_t e = error_word_ptr(&g.a.c.err);
    if (e == cudaSuccess) e = split(pr, &g.sp);
    if (e != cudaSuccess) return e;
    const PagedCache &c = pr.c;
    const Layout l = layout(pr, g.sp);
    char *base = static_cast<char *>(ws);
    g.s.z = reinterpret_cast<float *>(base);
    g.s.stats = reinterpret_cast<float2 *>(base + l.stats);
    g.s.sums = reinterpret_cast<float2 *>(base + l.sums);
    g.s.o = reinterpret_cast<float *>(base + l.o);
    g.s.next = reinterpret_cast<unsigned *>(base + l.counts);
    g.s.scored = g.s.next + 1;
    g.s.summed = g.s.scored + g.sp.rows;
    // a copy takes the rows of one page that lie in one tile: the largest power
    // of two that divides the page size, so that no copy crosses either border
    const int low = c.page_size & -c.page_size;
    g.piece_rows = low < paged::tile_keys(c.d) ? low : paged::tile_keys(c.d);
    CUtensorMap km, vm;
    if (!make_page_map(&km, c.k, c.half, c.d, c.Hkv * c.page_size, c.n_pages, c.page_stride, g.piece_rows) ||
        !make_page_map(&vm, c.v, c.half, c.d, c.Hkv * c.page_size, c.n_pages, c.page_stride, g.piece_rows))
        return cudaErrorInvalidValue;
    if ((e = cudaMemsetAsync(g.s.next, 0, l.total - l.counts, stream)) != cudaSuccess) return e;
    const auto launch = c.half ? (c.d == 64 ? paged::fp16_d64_launch : paged::fp16_d128_launch)
                               : (c.d == 64 ? paged::bf16_d64_launch : paged::bf16_d128_launch);
    return launch(km, vm, g, stream);
}

}  // namespace lssar
