// Paged cache, append: the new tokens' key and value rows go to their slots.
//
// Token t of sequence b (t < counts[b]) has slot lens[b] + t; its rows of
// every key head are copied to the slot's page, its added-up weight starts at
// 0 and its position is first[b] + t.  A copy: 4d bytes of each (token, head)
// are read and written once, so HBM bounds it.  Consecutive threads take
// consecutive 16-byte vectors of consecutive tokens of one head, which fill a
// page's rows of that head from front to back.
#include "paged.cuh"
#include "tc_host.cuh"

namespace lssar {
namespace {

constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) paged_append(const PagedAppend a) {
    const PagedCache &c = a.c;
    const long long idx = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
    if (idx < c.B) {   // the new lengths, by the first B threads
        const int b = (int)idx, cnt = a.counts ? a.counts[b] : a.n, len = c.lens[b];
        const bool ok = len >= 0 && cnt >= 0 && cnt <= a.n && (long long)len + cnt <= c.capacity();
        if (!ok) atomicCAS(c.err, 0u, (unsigned)kErrPagedLength);
        a.lens_out[b] = ok ? len + cnt : len;
    }
    const int parts = c.d / 8;
    const long long row = idx / parts;
    if (row >= (long long)c.B * c.Hkv * a.n) return;
    const int part = (int)(idx % parts);
    const int t = (int)(row % a.n), bh = (int)(row / a.n), b = bh / c.Hkv, h = bh % c.Hkv;
    const int cnt = a.counts ? a.counts[b] : a.n, len = c.lens[b];
    if (len < 0 || cnt < 0 || cnt > a.n || (long long)len + cnt > c.capacity() || t >= cnt) return;
    const int slot = len + t;
    if (part == 0) {
        const size_t at = (size_t)bh * c.capacity() + slot;
        if (a.scores) a.scores[at] = 0.f;
        if (a.positions) a.positions[at] = (a.first ? a.first[b] : len) + t;
    }
    const int pg = paged_page(c, b, slot / c.page_size);
    if (pg < 0) return;
    const auto *k = static_cast<const uint16_t *>(a.k_new) + b * a.ks[0] + h * a.ks[1] + t * a.ks[2] + part * 8;
    const auto *v = static_cast<const uint16_t *>(a.v_new) + b * a.vs[0] + h * a.vs[1] + t * a.vs[2] + part * 8;
    const uint4 kx = *reinterpret_cast<const uint4 *>(k), vx = *reinterpret_cast<const uint4 *>(v);
    const size_t to = pg * c.page_stride + ((size_t)h * c.page_size + slot % c.page_size) * c.d + part * 8;
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(c.k) + to) = kx;
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(c.v) + to) = vx;
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppend &pr, cudaStream_t stream) {
    PagedAppend a = pr;
    cudaError_t e = error_word_ptr(&a.c.err);
    if (e != cudaSuccess) return e;
    long long threads = (long long)a.c.B * a.c.Hkv * a.n * (a.c.d / 8);
    if (threads < a.c.B) threads = a.c.B;
    const long long blocks = (threads + kAppendThreads - 1) / kAppendThreads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    paged_append<<<(unsigned)blocks, kAppendThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace lssar
