// Host side of the paged decode: the split, the scratch layout and the launches.
#include "paged_decode.cuh"

namespace lssar {
namespace {

struct Layout {
    paged::Split sp;
    size_t stats, sums, o, total;   // z first
};

Layout layout(const PagedDecode &pr, int sms) {
    const PagedCache &c = pr.c;
    Layout l;
    paged::Split &sp = l.sp;
    sp.G = pr.H / c.Hkv;
    sp.blocks = (sp.G + paged::kHeads - 1) / paged::kHeads;
    sp.heads_rows = c.Hkv * sp.blocks;
    sp.zg = sp.G < paged::kHeads ? sp.G : paged::kHeads;
    const int keys = paged::tile_keys(c.d);
    const size_t rows = (size_t)c.B * sp.heads_rows, tiles = rows * ((c.capacity() + keys - 1) / keys);
    const size_t wave = (size_t)sms * (c.d == 64 ? paged::Config<64, paged::kValues>::kPerSm : paged::Config<128, paged::kValues>::kPerSm);
    sp.ctas = (int)(tiles < wave ? tiles : wave);
    const size_t segments = (rows + sp.ctas) * sp.zg;
    const bool reweight = is_reweight(pr.mode);
    auto r = [](size_t x) { return (x + 255) & ~(size_t)255; };
    l.stats = reweight || pr.scores ? r(tiles * sp.zg * keys * 4) : 0;
    l.sums = l.stats + (reweight ? r(segments * 8) : 0);
    l.o = l.sums + r(segments * 8);
    l.total = l.o + r(segments * c.d * 4);
    return l;
}

}  // namespace

size_t paged_decode_workspace_bytes(const PagedDecode &pr, int sms) { return layout(pr, sms).total; }

cudaError_t launch_paged_decode(const PagedDecode &pr, void *ws, int sms, cudaStream_t stream) {
    paged::Args g;
    g.a = pr;
    cudaError_t e = error_word_ptr(&g.a.c.err);
    if (e != cudaSuccess) return e;
    const PagedCache &c = pr.c;
    const Layout l = layout(pr, sms);
    g.sp = l.sp;
    char *base = static_cast<char *>(ws);
    g.s.z = reinterpret_cast<float *>(base);
    g.s.stats = reinterpret_cast<float2 *>(base + l.stats);
    g.s.sums = reinterpret_cast<float2 *>(base + l.sums);
    g.s.o = reinterpret_cast<float *>(base + l.o);
    // a copy takes the rows of one page that lie in one tile: the largest power
    // of two that divides the page size, so that no copy crosses either border
    const int low = c.page_size & -c.page_size;
    g.piece_rows = low < paged::tile_keys(c.d) ? low : paged::tile_keys(c.d);
    CUtensorMap km, vm;
    if (!make_page_map(&km, c.k, c.half, c.d, c.Hkv * c.page_size, c.n_pages, c.page_stride, g.piece_rows) ||
        !make_page_map(&vm, c.v, c.half, c.d, c.Hkv * c.page_size, c.n_pages, c.page_stride, g.piece_rows))
        return cudaErrorInvalidValue;
    const auto launch = c.half ? (c.d == 64 ? paged::fp16_d64_launch : paged::fp16_d128_launch)
                               : (c.d == 64 ? paged::bf16_d64_launch : paged::bf16_d128_launch);
    return launch(km, vm, g, sms, stream);
}

}  // namespace lssar
