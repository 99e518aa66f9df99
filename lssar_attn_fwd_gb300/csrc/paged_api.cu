// C ABI of the paged key-value cache: argument validation and dispatch.  The
// declarations and the full contract are in include/lssar_attn_fwd.h.
#include <cstdint>
#include <initializer_list>

#include "lssar_attn_fwd.h"
#include "paged.cuh"

namespace {

constexpr int kMaxPageSize = 256;
constexpr unsigned long long kMaxElems = 1ULL << 40;

// A stretch of device memory that a call reads or writes.
struct Range {
    const void *p;
    size_t bytes;
};

bool overlap(const Range &a, const Range &b) {
    const auto x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Checks of the cache description (pure host); fills *out.
int check_cache(const lssar_paged_cache_t *c, lssar::PagedCache *out) {
    if (!c || !c->k_pages || !c->v_pages || !c->table || !c->lens) return LSSAR_ERR_NULL;
    if (c->d != 64 && c->d != 128) return LSSAR_ERR_HEADDIM;
    if (c->dtype != LSSAR_DTYPE_BF16 && c->dtype != LSSAR_DTYPE_FP16) return LSSAR_ERR_DTYPE;
    if (c->B < 1 || c->Hkv < 1 || c->max_pages < 1) return LSSAR_ERR_SHAPE;
    if (c->page_size < 8 || c->page_size > kMaxPageSize || c->page_size % 8 || c->n_pages < 1) return LSSAR_ERR_PAGE;
    const unsigned long long block = (unsigned long long)c->Hkv * c->page_size * c->d;
    if (block > (1ULL << 31) || c->page_stride < (long long)block || c->page_stride % 8 ||
        (unsigned long long)c->page_stride > kMaxElems || (unsigned long long)c->n_pages * c->page_stride > kMaxElems)
        return LSSAR_ERR_PAGE;
    const unsigned long long cap = (unsigned long long)c->max_pages * c->page_size;
    if (cap > (1ULL << 24) || (unsigned long long)c->B * c->Hkv > (1ULL << 24) ||
        (unsigned long long)c->B * c->Hkv * cap * c->d > kMaxElems)
        return LSSAR_ERR_SHAPE;
    if (misaligned(c->k_pages, 16) || misaligned(c->v_pages, 16) || misaligned(c->table, 4) || misaligned(c->lens, 4))
        return LSSAR_ERR_ALIGN;
    // K and V may be interleaved in one buffer, page by page: their blocks of
    // `block` elements, page_stride apart, must not meet
    const long long bytes = (long long)block * 2, stride = c->page_stride * 2;
    const long long gap = (long long)(reinterpret_cast<intptr_t>(c->v_pages) - reinterpret_cast<intptr_t>(c->k_pages));
    const long long span = (c->n_pages - 1) * stride + bytes;
    if (gap > -span && gap < span) {
        const long long r = ((gap % stride) + stride) % stride;
        if (r < bytes || r > stride - bytes) return LSSAR_ERR_ALIAS;
    }
    *out = lssar::PagedCache{c->k_pages, c->v_pages, c->table, c->lens, c->page_stride, c->n_pages, c->max_pages,
                             c->page_size, c->B, c->Hkv, c->d, c->dtype == LSSAR_DTYPE_FP16, nullptr};
    return LSSAR_OK;
}

// Bytes from the first page of K or V to the end of the last.
size_t page_bytes(const lssar::PagedCache &c) {
    return ((size_t)(c.n_pages - 1) * c.page_stride + (size_t)c.Hkv * c.page_size * c.d) * 2;
}

// The memory of K, V, table and lens, with `outs` (written) tested against
// them, against one another and against `ins` (read).
bool any_alias(const lssar::PagedCache &c, std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    const size_t pages = page_bytes(c);
    const Range own[4] = {{c.k, pages}, {c.v, pages}, {c.table, (size_t)c.B * c.max_pages * 4}, {c.lens, (size_t)c.B * 4}};
    for (const Range *o = outs.begin(); o != outs.end(); ++o) {
        for (const Range &x : own)
            if (overlap(*o, x)) return true;
        for (const Range &x : ins)
            if (overlap(*o, x)) return true;
        for (const Range *x = outs.begin(); x != o; ++x)
            if (overlap(*o, *x)) return true;
    }
    return false;
}

// A [B, Hkv, n, d] view by its strides in elements: the innermost dimension is
// contiguous, the others any multiple of 8 (16-byte rows).  Fills the range it spans.
int check_view(const void *p, const long long *s, long long B, long long H, long long n, int d, Range *r) {
    unsigned long long last = 0;
    const long long dims[3] = {B, H, n};
    for (int i = 0; i < 3; ++i) {
        if (s[i] < 0 || s[i] > (long long)kMaxElems) return LSSAR_ERR_SHAPE;
        if (dims[i] > 1 && s[i] % 8) return LSSAR_ERR_ALIGN;
        last += (unsigned long long)(dims[i] > 0 ? dims[i] - 1 : 0) * s[i];
        if (last > kMaxElems) return LSSAR_ERR_SHAPE;
    }
    if (misaligned(p, 16)) return LSSAR_ERR_ALIGN;
    *r = Range{p, (size_t)(last + d) * 2};
    return LSSAR_OK;
}

}  // namespace

extern "C" {

int lssar_paged_append(const lssar_paged_cache_t *cache, const void *k_new, const long long *k_strides,
                       const void *v_new, const long long *v_strides, int n, const int *counts,
                       const int *first_positions, float *scores, int *positions, int *lens_out, cudaStream_t stream) {
    lssar::PagedAppend a = {};
    int st = check_cache(cache, &a.c);
    if (st != LSSAR_OK) return st;
    if (!lens_out || !k_strides || !v_strides || (n != 0 && (!k_new || !v_new))) return LSSAR_ERR_NULL;
    if (n < 0 || n > (1 << 24) || (unsigned long long)a.c.B * a.c.Hkv * n > (1ULL << 31)) return LSSAR_ERR_SHAPE;
    Range kr = {nullptr, 0}, vr = {nullptr, 0};
    if (n > 0) {
        if ((st = check_view(k_new, k_strides, a.c.B, a.c.Hkv, n, a.c.d, &kr)) != LSSAR_OK) return st;
        if ((st = check_view(v_new, v_strides, a.c.B, a.c.Hkv, n, a.c.d, &vr)) != LSSAR_OK) return st;
    }
    for (const void *p : {(const void *)counts, (const void *)first_positions, (const void *)scores,
                          (const void *)positions, (const void *)lens_out})
        if (misaligned(p, 4)) return LSSAR_ERR_ALIGN;
    const size_t slots = (size_t)a.c.B * a.c.Hkv * a.c.capacity() * 4, seqs = (size_t)a.c.B * 4;
    const Range sc = {scores, slots}, po = {positions, slots}, lo = {lens_out, seqs};
    const Range cn = {counts, seqs}, fi = {first_positions, seqs};
    if (any_alias(a.c, {sc, po, lo}, {kr, vr, cn, fi})) return LSSAR_ERR_ALIAS;
    // the pages are written too (table, lens and the inputs are read, and may be the same)
    for (const Range &r : {kr, vr, cn, fi})
        if (overlap(r, {a.c.k, page_bytes(a.c)}) || overlap(r, {a.c.v, page_bytes(a.c)})) return LSSAR_ERR_ALIAS;
    a.k_new = k_new;
    a.v_new = v_new;
    for (int i = 0; i < 3; ++i) {
        a.ks[i] = k_strides[i];
        a.vs[i] = v_strides[i];
    }
    a.n = n;
    a.counts = counts;
    a.first = first_positions;
    a.scores = scores;
    a.positions = positions;
    a.lens_out = lens_out;
    return lssar::launch_paged_append(a, stream) == cudaSuccess ? LSSAR_OK : LSSAR_ERR_CUDA;
}

int lssar_paged_decode(const lssar_paged_cache_t *cache, const void *q, const long long *q_strides, void *out, int H,
                       int p, int mode, const float *scores, float *scores_out, cudaStream_t stream) {
    lssar::PagedDecode a = {};
    int st = check_cache(cache, &a.c);
    if (st != LSSAR_OK) return st;
    if (!q || !q_strides || !out || !scores != !scores_out) return LSSAR_ERR_NULL;
    if (mode < LSSAR_MODE_SOFTMAX || mode > LSSAR_MODE_SIGMOID_RW) return LSSAR_ERR_MODE;
    // (tile numbers are ints, and the CTAs' first tiles reach up to one CTA's count past the last)
    if (H < 1 || H % a.c.Hkv || H / a.c.Hkv > 128 || (unsigned long long)a.c.B * H > (1ULL << 24) ||
        (unsigned long long)a.c.B * a.c.Hkv * ((H / a.c.Hkv + 7) / 8) * ((a.c.capacity() + 63) / 64) > 0x7fff0000ULL)
        return LSSAR_ERR_SHAPE;
    const bool reweight = lssar::is_reweight(mode);
    if (reweight && (p < 1 || p > 1024)) return LSSAR_ERR_P;
    const long long strides[3] = {q_strides[0], q_strides[1], 0};
    Range qr;
    if ((st = check_view(q, strides, a.c.B, H, 1, a.c.d, &qr)) != LSSAR_OK) return st;
    if (misaligned(out, 16) || misaligned(scores, 4) || misaligned(scores_out, 4)) return LSSAR_ERR_ALIGN;
    const size_t slots = (size_t)a.c.B * a.c.Hkv * a.c.capacity() * 4;
    const Range orow = {out, (size_t)a.c.B * H * a.c.d * 2}, so = {scores_out, slots}, si = {scores, slots};
    if (any_alias(a.c, {orow, so}, {qr}) || overlap(orow, si) || (scores != scores_out && overlap(so, si)))
        return LSSAR_ERR_ALIAS;
    a.q = q;
    a.q_b = q_strides[0];
    a.q_h = q_strides[1];
    a.out = out;
    a.H = H;
    a.p = reweight ? p : 1;
    a.mode = mode;
    a.scores = scores;
    a.scores_out = scores_out;
    int sms = 0;
    if (lssar::device_sms(&sms) != cudaSuccess) return LSSAR_ERR_CUDA;
    void *ws = nullptr;
    if (lssar::scratch_alloc(&ws, lssar::paged_decode_workspace_bytes(a, sms), stream) != cudaSuccess) return LSSAR_ERR_CUDA;
    const cudaError_t e = lssar::launch_paged_decode(a, ws, sms, stream);
    if (cudaFreeAsync(ws, stream) != cudaSuccess) return LSSAR_ERR_CUDA;
    return e == cudaSuccess ? LSSAR_OK : LSSAR_ERR_CUDA;
}

int lssar_paged_evict(const lssar_paged_cache_t *cache, const float *scores, const int *positions, int keep, int recent,
                      int sinks, float *scores_out, int *positions_out, int *lens_out, cudaStream_t stream) {
    lssar::PagedEvict a = {};
    const int st = check_cache(cache, &a.c);
    if (st != LSSAR_OK) return st;
    if (!scores || !positions || !scores_out || !positions_out || !lens_out) return LSSAR_ERR_NULL;
    if (keep < 1 || recent < 0 || sinks < 0 || (long long)recent + sinks > keep) return LSSAR_ERR_KEEP;
    for (const void *p : {(const void *)scores, (const void *)positions, (const void *)scores_out,
                          (const void *)positions_out, (const void *)lens_out})
        if (misaligned(p, 4)) return LSSAR_ERR_ALIGN;
    const size_t slots = (size_t)a.c.B * a.c.Hkv * a.c.capacity() * 4;
    const Range si = {scores, slots}, pi = {positions, slots}, so = {scores_out, slots}, po = {positions_out, slots},
                lo = {lens_out, (size_t)a.c.B * 4};
    // in place (both outputs their own inputs) or apart
    if ((scores == scores_out) != (positions == positions_out)) return LSSAR_ERR_ALIAS;
    const bool in_place = scores == scores_out;
    if (any_alias(a.c, {so, po, lo}, {}) || any_alias(a.c, {si}, {pi}) || any_alias(a.c, {pi}, {}) || overlap(lo, si) ||
        overlap(lo, pi) ||
        (!in_place && (overlap(so, si) || overlap(so, pi) || overlap(po, si) || overlap(po, pi))))
        return LSSAR_ERR_ALIAS;
    a.scores = scores;
    a.positions = positions;
    a.scores_out = scores_out;
    a.positions_out = positions_out;
    a.lens_out = lens_out;
    a.keep = keep < a.c.capacity() ? keep : a.c.capacity();
    a.recent = recent;
    a.sinks = sinks;
    void *ws = nullptr;
    if (lssar::scratch_alloc(&ws, lssar::paged_evict_workspace_bytes(a), stream) != cudaSuccess) return LSSAR_ERR_CUDA;
    const cudaError_t e = lssar::launch_paged_evict(a, ws, stream);
    if (cudaFreeAsync(ws, stream) != cudaSuccess) return LSSAR_ERR_CUDA;
    return e == cudaSuccess ? LSSAR_OK : LSSAR_ERR_CUDA;
}

}  // extern "C"
