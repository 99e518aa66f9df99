// C ABI of the paged key-value cache: argument validation and dispatch.  The
// declarations and the full contract are in include/lssar_attn_fwd.h.
#include <initializer_list>

#include "api_checks.cuh"

using lssar::any_alias;
using lssar::check_cache;
using lssar::check_view;
using lssar::misaligned;
using lssar::overlap;
using lssar::page_bytes;
using lssar::Range;

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

int lssar_paged_append_rope(const lssar_paged_cache_t *cache, const void *q, const long long *q_strides, void *q_out,
                            int H, const void *k_new, const long long *k_strides, const void *v_new,
                            const long long *v_strides, int n, const lssar_rotary_t *rotary, const int *counts,
                            const int *first_positions, float *scores, int *positions, int *lens_out,
                            cudaStream_t stream) {
    lssar::PagedAppendRope r = {};
    lssar::PagedAppend &a = r.a;
    int st = check_cache(cache, &a.c);
    if (st != LSSAR_OK) return st;
    if (!lens_out || !q_strides || !k_strides || !v_strides || (n != 0 && (!q || !q_out || !k_new || !v_new))) return LSSAR_ERR_NULL;
    if (n < 0 || n > (1 << 24) || H < 1 || H > (1 << 24) || (unsigned long long)a.c.B * a.c.Hkv * n > (1ULL << 31) ||
        (unsigned long long)a.c.B * H * n > (1ULL << 31))
        return LSSAR_ERR_SHAPE;
    if ((st = lssar::rotary_table(rotary, a.c.d, &r.table)) != LSSAR_OK) return st;
    Range kr = {}, vr = {}, qr = {}, qo = {};
    if (n > 0) {
        if ((st = check_view(k_new, k_strides, a.c.B, a.c.Hkv, n, a.c.d, &kr)) != LSSAR_OK) return st;
        if ((st = check_view(v_new, v_strides, a.c.B, a.c.Hkv, n, a.c.d, &vr)) != LSSAR_OK) return st;
        if ((st = lssar::rope_view(q, q_strides, q_out, a.c.B, H, n, a.c.d, &r.q, &qr, &qo)) != LSSAR_OK) return st;
    }
    for (const void *p : {(const void *)counts, (const void *)first_positions, (const void *)scores,
                          (const void *)positions, (const void *)lens_out})
        if (misaligned(p, 4)) return LSSAR_ERR_ALIGN;
    const size_t slots = (size_t)a.c.B * a.c.Hkv * a.c.capacity() * 4, seqs = (size_t)a.c.B * 4;
    const Range sc = {scores, slots}, po = {positions, slots}, lo = {lens_out, seqs};
    const Range cn = {counts, seqs}, fi = {first_positions, seqs};
    const bool in_place = q == q_out;
    if (any_alias(a.c, {sc, po, lo}, {kr, vr, cn, fi, qr}) || any_alias(a.c, {sc, po, lo, qo}, {cn, fi})) return LSSAR_ERR_ALIAS;
    if (!in_place && overlap(qo, qr)) return LSSAR_ERR_ALIAS;
    if (overlap(qo, kr) && !(in_place && lssar::slices_apart(q_strides, q, H, k_strides, k_new, a.c.Hkv, a.c.B, n, a.c.d))) return LSSAR_ERR_ALIAS;
    if (overlap(qo, vr) && !(in_place && lssar::slices_apart(q_strides, q, H, v_strides, v_new, a.c.Hkv, a.c.B, n, a.c.d))) return LSSAR_ERR_ALIAS;
    for (const Range &x : {kr, vr, cn, fi, qr})
        if (overlap(x, {a.c.k, page_bytes(a.c)}) || overlap(x, {a.c.v, page_bytes(a.c)})) return LSSAR_ERR_ALIAS;
    a.k_new = k_new;
    a.v_new = v_new;
    for (int i = 0; i < 3; ++i) {
        a.ks[i] = k_strides[i];
        a.vs[i] = v_strides[i];
    }
    r.q.H = H;
    a.n = n;
    a.counts = counts;
    a.first = first_positions;
    a.scores = scores;
    a.positions = positions;
    a.lens_out = lens_out;
    return lssar::launch_paged_append_rope(r, stream) == cudaSuccess ? LSSAR_OK : LSSAR_ERR_CUDA;
}

int lssar_paged_attend(const lssar_paged_cache_t *cache, const void *q, const long long *q_strides, void *out, int H,
                       int n, const int *counts, int p, int mode, cudaStream_t stream) {
    lssar::PagedAttend a = {};
    int st = check_cache(cache, &a.c);
    if (st != LSSAR_OK) return st;
    if (!q || !q_strides || !out) return LSSAR_ERR_NULL;
    if (mode < LSSAR_MODE_SOFTMAX || mode > LSSAR_MODE_SIGMOID_RW) return LSSAR_ERR_MODE;
    if (H < 1 || H % a.c.Hkv || H / a.c.Hkv > 128 || n < 1 || n > (1 << 24) ||
        (unsigned long long)a.c.B * H * n > (1ULL << 31))
        return LSSAR_ERR_SHAPE;
    const bool reweight = lssar::is_reweight(mode);
    if (reweight && (p < 1 || p > 1024)) return LSSAR_ERR_P;
    Range qr;
    if ((st = check_view(q, q_strides, a.c.B, H, n, a.c.d, &qr)) != LSSAR_OK) return st;
    if (misaligned(out, 16) || misaligned(counts, 4)) return LSSAR_ERR_ALIGN;
    a.H = H;
    a.n = n;
    // (tile numbers are ints, and the CTAs' first tiles reach up to one CTA's count past the last)
    if (lssar::paged_attend_tiles(a) > 0x7fff0000LL) return LSSAR_ERR_SHAPE;
    const Range orow = {out, (size_t)a.c.B * H * n * a.c.d * 2}, cn = {counts, (size_t)a.c.B * 4};
    if (any_alias(a.c, {orow}, {qr, cn})) return LSSAR_ERR_ALIAS;
    a.q = q;
    for (int i = 0; i < 3; ++i) a.qs[i] = q_strides[i];
    a.out = out;
    a.counts = counts;
    a.p = reweight ? p : 1;
    a.mode = mode;
    int sms = 0;
    if (lssar::device_sms(&sms) != cudaSuccess) return LSSAR_ERR_CUDA;
    void *ws = nullptr;
    const size_t bytes = lssar::paged_attend_workspace_bytes(a, sms);
    if (bytes && lssar::scratch_alloc(&ws, bytes, stream) != cudaSuccess) return LSSAR_ERR_CUDA;
    const cudaError_t e = lssar::launch_paged_attend(a, ws, sms, stream);
    if (ws && cudaFreeAsync(ws, stream) != cudaSuccess) return LSSAR_ERR_CUDA;
    return e == cudaSuccess ? LSSAR_OK : LSSAR_ERR_CUDA;
}

// Sizes and pointers that reserve and release share.
static int check_pages(const lssar::PagedPages &a, bool reserve) {
    if (!a.table || !a.lens || (!reserve && !a.other) || !a.free_pages || !a.free_count || !a.free_out || (reserve && !a.counts_out))
        return LSSAR_ERR_NULL;
    if (a.B < 1 || a.B > (1 << 24) || a.max_pages < 1) return LSSAR_ERR_SHAPE;
    if (a.page_size < 8 || a.page_size > lssar::kMaxPageSize || a.page_size % 8 || a.n_pages < 1) return LSSAR_ERR_PAGE;
    if ((unsigned long long)a.max_pages * a.page_size > (1ULL << 24)) return LSSAR_ERR_SHAPE;
    for (const void *p : {(const void *)a.table, (const void *)a.lens, (const void *)a.other, (const void *)a.free_pages,
                          (const void *)a.free_count, (const void *)a.counts_out, (const void *)a.free_out})
        if (misaligned(p, 4)) return LSSAR_ERR_ALIGN;
    const size_t seqs = (size_t)a.B * 4;
    const Range table = {a.table, seqs * a.max_pages}, list = {a.free_pages, (size_t)a.n_pages * 4}, count = {a.free_count, 4};
    const Range lens = {a.lens, seqs}, other = {a.other, seqs}, counts_out = {a.counts_out, seqs}, free_out = {a.free_out, 4};
    const Range written[3] = {reserve ? table : list, counts_out, free_out}, read[4] = {reserve ? list : table, count, lens, other};
    for (int i = 0; i < 3; ++i) {
        for (const Range &x : read)
            if (overlap(written[i], x)) return LSSAR_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(written[i], written[j])) return LSSAR_ERR_ALIAS;
    }
    return LSSAR_OK;
}

int lssar_paged_reserve(int *table, int max_pages, int page_size, const int *lens, const int *counts, int B,
                        const int *free_pages, int n_pages, const int *free_count, int *counts_out, int *free_out,
                        cudaStream_t stream) {
    const lssar::PagedPages a = {table, lens, counts, const_cast<int *>(free_pages), free_count, counts_out, free_out,
                                 B, max_pages, page_size, n_pages, nullptr};
    const int st = check_pages(a, true);
    if (st != LSSAR_OK) return st;
    return lssar::launch_paged_reserve(a, stream) == cudaSuccess ? LSSAR_OK : LSSAR_ERR_CUDA;
}

int lssar_paged_release(const int *table, int max_pages, int page_size, const int *lens, const int *lens_new, int B,
                        int *free_pages, int n_pages, const int *free_count, int *free_out, cudaStream_t stream) {
    const lssar::PagedPages a = {const_cast<int *>(table), lens, lens_new, free_pages, free_count, nullptr, free_out,
                                 B, max_pages, page_size, n_pages, nullptr};
    const int st = check_pages(a, false);
    if (st != LSSAR_OK) return st;
    return lssar::launch_paged_release(a, stream) == cudaSuccess ? LSSAR_OK : LSSAR_ERR_CUDA;
}

}  // extern "C"
