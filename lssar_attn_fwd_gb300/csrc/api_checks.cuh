// Argument checks shared by the C entry points of the paged cache and of the
// rotary positions (pure host).
#pragma once

#include <cstdint>
#include <initializer_list>
#include <utility>

#include "lssar_attn_fwd.h"
#include "paged.cuh"
#include "rope.cuh"

namespace lssar {

constexpr int kMaxPageSize = 256;
constexpr unsigned long long kMaxElems = 1ULL << 40;

// A stretch of device memory that a call reads or writes.
struct Range {
    const void *p;
    size_t bytes;
};

inline bool overlap(const Range &a, const Range &b) {
    const auto x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

inline bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Checks of the cache description (pure host); fills *out.
inline int check_cache(const lssar_paged_cache_t *c, PagedCache *out) {
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
    *out = PagedCache{c->k_pages, c->v_pages, c->table, c->lens, c->page_stride, c->n_pages, c->max_pages,
                             c->page_size, c->B, c->Hkv, c->d, c->dtype == LSSAR_DTYPE_FP16, nullptr};
    return LSSAR_OK;
}

// Bytes from the first page of K or V to the end of the last.
inline size_t page_bytes(const PagedCache &c) {
    return ((size_t)(c.n_pages - 1) * c.page_stride + (size_t)c.Hkv * c.page_size * c.d) * 2;
}

// The memory of K, V, table and lens, with `outs` (written) tested against
// them, against one another and against `ins` (read).
inline bool any_alias(const PagedCache &c, std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
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
inline int check_view(const void *p, const long long *s, long long B, long long H, long long n, int d, Range *r) {
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

// Whether no two rows of d elements of a [B, H, n, d] view overlap: taken by their strides,
// from the smallest on, each dimension steps over what those before it span.
inline bool rows_apart(const long long *s, long long B, long long H, long long n, int d) {
    long long dims[3] = {B, H, n}, st[3] = {s[0], s[1], s[2]}, span = d;
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                std::swap(st[i], st[j]);
                std::swap(dims[i], dims[j]);
            }
    for (int i = 0; i < 3; ++i) {
        if (dims[i] <= 1) continue;
        if (st[i] < span) return false;
        span += (dims[i] - 1) * st[i];
    }
    return true;
}

// Whether two views [B, Hx, n, d] and [B, Hy, n, d] are slices of the heads of one buffer
// that do not meet: equal strides of (B, n), and the heads of a token apart modulo them.
inline bool slices_apart(const long long *xs, const void *x, long long Hx, const long long *ys, const void *y, long long Hy,
                         long long B, long long n, int d) {
    if ((n > 1 && xs[2] != ys[2]) || (B > 1 && xs[0] != ys[0])) return false;
    const long long delta = (long long)(reinterpret_cast<intptr_t>(y) - reinterpret_cast<intptr_t>(x)) / 2;
    const long long a = (Hx - 1) * xs[1] + d, b = (Hy - 1) * ys[1] + d;
    if (n <= 1 && B <= 1) return delta >= a || -delta >= b;
    const long long m = n > 1 ? xs[2] : xs[0];
    if (m < 1 || (n > 1 && B > 1 && xs[0] % m)) return false;
    const long long r = ((delta % m) + m) % m;
    return r >= a && r + b <= m;
}

// A tensor that turns, x -> y: y contiguous, or x itself (in place, at its own strides).
inline int rope_view(const void *x, const long long *s, void *y, int B, int H, int n, int d, RopeView *v, Range *in, Range *out) {
    const int st = check_view(x, s, B, H, n, d, in);
    if (st != LSSAR_OK) return st;
    if (misaligned(y, 16)) return LSSAR_ERR_ALIGN;
    v->x = static_cast<const uint16_t *>(x);
    v->y = static_cast<uint16_t *>(y);
    v->H = H;
    const bool in_place = x == y;
    if (in_place && !rows_apart(s, B, H, n, d)) return LSSAR_ERR_ALIAS;
    const long long whole[3] = {(long long)H * n * d, (long long)n * d, d};
    for (int i = 0; i < 3; ++i) {
        v->xs[i] = s[i];
        v->ys[i] = in_place ? s[i] : whole[i];
    }
    *out = in_place ? *in : Range{y, (size_t)B * H * n * d * 2};
    return LSSAR_OK;
}

}  // namespace lssar
