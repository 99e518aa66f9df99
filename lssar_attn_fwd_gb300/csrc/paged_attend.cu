// Host side of the chunk attention: the split, the scratch layout and the launches.
#include "paged_attend.cuh"

namespace lssar {
namespace {

struct Layout {
    int G, tokens, ctas, rows, cap128;
    size_t entries, first, knorm, stats, sums, o, total;   // the header first
};

Layout layout(const PagedAttend &pr, int sms) {
    const PagedCache &c = pr.c;
    Layout l;
    l.G = pr.H / c.Hkv;
    l.tokens = attend::kPairRows / l.G;
    l.rows = (pr.n < l.tokens ? pr.n : l.tokens) * l.G;
    l.cap128 = (c.capacity() + attend::kKeys - 1) / attend::kKeys * attend::kKeys;
    const size_t pairs = (size_t)c.B * ((pr.n + l.tokens - 1) / l.tokens), items = pairs * c.Hkv, tiles = items * (2 * (l.cap128 / attend::kKeys) + attend::kItemCost);
    l.ctas = (int)(tiles < (size_t)sms ? tiles : sms);
    const bool norms = uses_normalised_qk(pr.mode), reweight = is_reweight(pr.mode);
    auto r = [](size_t x) { return (x + 255) & ~(size_t)255; };
    l.entries = 256;
    l.first = l.entries + r(pairs * sizeof(int4));
    l.knorm = l.first + r((size_t)l.ctas * 2 * sizeof(int4));
    l.stats = l.knorm + (norms ? r((size_t)c.B * c.Hkv * l.cap128 * 4) : 0);
    l.sums = l.stats + (reweight ? r((items + l.ctas) * l.rows * 8) : 0);
    l.o = l.sums + r((size_t)2 * l.ctas * l.rows * 8);
    l.total = l.o + r((size_t)2 * l.ctas * l.rows * c.d * 4);
    return l;
}

}  // namespace

long long paged_attend_tiles(const PagedAttend &pr) {
    const long long tokens = attend::kPairRows / (pr.H / pr.c.Hkv), pairs = (pr.n + tokens - 1) / tokens;
    const long long tiles = (pr.c.capacity() + 63) / 64 + 1 + attend::kItemCost;      // units of cost of an item (at least the prologue's tiles)
    return (long long)pr.c.B * pr.c.Hkv * pairs > (1LL << 31) ? 1LL << 62 : (long long)pr.c.B * pr.c.Hkv * pairs * tiles;
}

size_t paged_attend_workspace_bytes(const PagedAttend &pr, int sms) { return layout(pr, sms).total; }

cudaError_t launch_paged_attend(const PagedAttend &pr, void *ws, int sms, cudaStream_t stream) {
    attend::Args g;
    g.a = pr;
    const cudaError_t e = error_word_ptr(&g.a.c.err);
    if (e != cudaSuccess) return e;
    const PagedCache &c = pr.c;
    const Layout l = layout(pr, sms);
    char *base = static_cast<char *>(ws);
    g.s.head = reinterpret_cast<attend::Header *>(base);
    g.s.entries = reinterpret_cast<int4 *>(base + l.entries);
    g.s.first = reinterpret_cast<int4 *>(base + l.first);
    g.s.knorm = reinterpret_cast<float *>(base + l.knorm);
    g.s.stats = reinterpret_cast<float2 *>(base + l.stats);
    g.s.sums = reinterpret_cast<float2 *>(base + l.sums);
    g.s.o = reinterpret_cast<float *>(base + l.o);
    g.G = l.G;
    g.tokens = l.tokens;
    g.ctas = l.ctas;
    g.rows = l.rows;
    g.cap128 = l.cap128;
    // a copy takes the rows of one page that lie in one tile: the largest power
    // of two that divides the page size, so that no copy crosses either border
    const int low = c.page_size & -c.page_size;
    g.piece_rows = low < attend::kKeys ? low : attend::kKeys;
    g.scale = !uses_normalised_qk(pr.mode) ? 1.4426950408889634f / sqrtf((float)c.d) : (pr.mode == kSigmoidRw ? -1.f : 1.f) * score_qmul(c.d);
    g.exact_weights = exact_weights_requested() ? 1 : 0;
    g.power = {pr.p, 0, pr.p};
    for (; g.power.rest % 3 == 0; g.power.rest /= 3) ++g.power.cubes;
    g.idesc_s = ptx::idesc_f16(!c.half, attend::kTileRows, attend::kKeys, false, false);
    g.idesc_s64 = ptx::idesc_f16(!c.half, attend::kTileRows, 64, false, false);
    g.idesc_pv = ptx::idesc_f16(!c.half, attend::kTileRows, c.d, false, true);
    CUtensorMap km, vm;
    if (!make_group_map(&km, c.k, c.half, c.d, c.Hkv * c.page_size, c.n_pages, c.page_stride, g.piece_rows) ||
        !make_group_map(&vm, c.v, c.half, c.d, c.Hkv * c.page_size, c.n_pages, c.page_stride, g.piece_rows))
        return cudaErrorInvalidValue;
    using namespace attend;
    Launch *const launch[5][2] = {{softmax_d64, softmax_d128}, {lssa_d64, lssa_d128}, {lssar_d64, lssar_d128},
                                  {softmax_rw_d64, softmax_rw_d128}, {sigmoid_rw_d64, sigmoid_rw_d128}};
    return launch[pr.mode][c.d == 128](km, vm, g, sms, stream);
}

}  // namespace lssar
