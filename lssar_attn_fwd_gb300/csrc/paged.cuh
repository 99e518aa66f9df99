// Internal declarations of the paged key-value cache: append, decode, evict.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "lssar_internal.cuh"

namespace lssar {

// device error word codes of the paged kernels (51 and 52 are the caller's
// data, read on the device; the others are waits that gave up)
enum : unsigned { kErrPagedLength = 51, kErrPagedPage = 52 };

// The cache as the kernels see it; checked by the host as far as the host can
// see (not the contents of table and lens, which the kernels check).
// Element (page, h, r, c) of K or V lies at page * page_stride + (h * page_size + r) * d + c.
struct PagedCache {
    void *k, *v;         // 16-bit elements
    const int *table;    // [B, max_pages]
    const int *lens;     // [B]
    long long page_stride;
    int n_pages, max_pages, page_size, B, Hkv, d;
    bool half;           // fp16, else bf16
    unsigned *err;
    __host__ __device__ int capacity() const { return max_pages * page_size; }
};

struct PagedAppend {
    PagedCache c;
    const void *k_new, *v_new;
    long long ks[3], vs[3];   // element strides of (b, h, t)
    int n;
    const int *counts, *first;   // [B] or null
    float *scores;               // [B, Hkv, capacity] or null
    int *positions;              // [B, Hkv, capacity] or null
    int *lens_out;               // [B]
};
cudaError_t launch_paged_append(const PagedAppend &pr, cudaStream_t stream);

struct PagedDecode {
    PagedCache c;
    const void *q;            // (b, h) rows at q_b * b + q_h * h
    long long q_b, q_h;
    void *out;                // [B, H, d]
    int H, p, mode;
    const float *scores;      // [B, Hkv, capacity] or null
    float *scores_out;
};
size_t paged_decode_workspace_bytes(const PagedDecode &pr, int sms);
cudaError_t launch_paged_decode(const PagedDecode &pr, void *ws, int sms, cudaStream_t stream);

struct PagedEvict {
    PagedCache c;
    const float *scores;      // [B, Hkv, capacity]
    const int *positions;
    float *scores_out;
    int *positions_out, *lens_out;
    int keep, recent, sinks;
};
size_t paged_evict_workspace_bytes(const PagedEvict &pr);
cudaError_t launch_paged_evict(const PagedEvict &pr, void *ws, cudaStream_t stream);

// The length of sequence b, or 0 with the error word set where it is outside
// 0..capacity.
__device__ __forceinline__ int paged_len(const PagedCache &c, int b) {
    const int n = c.lens[b];
    if (n >= 0 && n <= c.capacity()) return n;
    atomicCAS(c.err, 0u, (unsigned)kErrPagedLength);
    return 0;
}

// The page that holds page number i of sequence b, or -1 with the error word
// set where the table's entry is no page of the pool.
__device__ __forceinline__ int paged_page(const PagedCache &c, int b, int i) {
    const int pg = c.table[(size_t)b * c.max_pages + i];
    if (pg >= 0 && pg < c.n_pages) return pg;
    atomicCAS(c.err, 0u, (unsigned)kErrPagedPage);
    return -1;
}

}  // namespace lssar
