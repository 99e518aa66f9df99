// Paged cache, append: the new tokens' key and value rows go to their slots.
//
// Token t of sequence b (t < counts[b]) has slot lens[b] + t; its rows of
// every key head are copied to the slot's page, its added-up weight starts at
// 0 and its position is first[b] + t.  A copy: 4d bytes of each (token, head)
// are read and written once, so HBM bounds it.  A block takes a stretch of
// tokens of one (sequence, head), which fills the rows of that head in its pages
// from front to back; d / 8 threads take a row, four rows of a group at once, so
// that their loads are in flight together.  Measured: one token for each of 8 sequences
// 4.2 us (a launch), 8 sequences of 32K tokens (1.07 GB read, as much written)
// 320 us, 99 % of the rate of a plain copy.
#include "paged.cuh"
#include "tc_host.cuh"

namespace lssar {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kRowsAtOnce = 4;

// `stretch`: tokens per block.
__global__ void __launch_bounds__(kAppendThreads) paged_append(const __grid_constant__ PagedAppend a, int stretch, int stretches) {
    const PagedCache &c = a.c;
    const int bh = blockIdx.x / stretches, b = bh / c.Hkv, h = bh - b * c.Hkv, t0 = (blockIdx.x - bh * stretches) * stretch;
    const int cnt = a.counts ? a.counts[b] : a.n, len = c.lens[b];
    const bool ok = len >= 0 && cnt >= 0 && cnt <= a.n && (long long)len + cnt <= c.capacity();
    if (h == 0 && t0 == 0 && threadIdx.x == 0) {
        if (!ok) atomicCAS(c.err, 0u, (unsigned)kErrPagedLength);
        a.lens_out[b] = ok ? len + cnt : len;
    }
    const int t1 = ok ? min(cnt, t0 + stretch) : 0;
    if (t0 >= t1) return;
    if (!dcheck(b < c.B && t0 >= 0 && len + t1 <= c.capacity(), c.err, kDbgItem)) return;
    const size_t at = (size_t)bh * c.capacity() + len;
    if (a.scores)
        for (int t = t0 + threadIdx.x; t < t1; t += kAppendThreads) a.scores[at + t] = 0.f;
    if (a.positions) {
        const int first = a.first ? a.first[b] : len;
        for (int t = t0 + threadIdx.x; t < t1; t += kAppendThreads) a.positions[at + t] = first + t;
    }
    const int parts = c.d / 8, part = threadIdx.x % parts, groups = kAppendThreads / parts;
    const uint16_t *k = static_cast<const uint16_t *>(a.k_new) + b * a.ks[0] + h * a.ks[1] + part * 8;
    const uint16_t *v = static_cast<const uint16_t *>(a.v_new) + b * a.vs[0] + h * a.vs[1] + part * 8;
    const int *table = c.table + (size_t)b * c.max_pages;
    bool bad = false;
#pragma unroll 1
    for (int t = t0 + threadIdx.x / parts; t < t1; t += kRowsAtOnce * groups) {
        uint4 kx[kRowsAtOnce], vx[kRowsAtOnce];
        int pg[kRowsAtOnce], row[kRowsAtOnce];
#pragma unroll
        for (int e = 0; e < kRowsAtOnce; ++e) {
            const int te = t + e * groups, i = (len + te) / c.page_size;
            pg[e] = 0;
            row[e] = len + te - i * c.page_size;
            if (te >= t1) continue;
            kx[e] = __ldcs(reinterpret_cast<const uint4 *>(k + te * a.ks[2]));
            vx[e] = __ldcs(reinterpret_cast<const uint4 *>(v + te * a.vs[2]));
            pg[e] = table[i];
        }
#pragma unroll
        for (int e = 0; e < kRowsAtOnce; ++e) {
            if (t + e * groups >= t1) continue;
            if ((unsigned)pg[e] >= (unsigned)c.n_pages) {
                bad = true;
                continue;
            }
            if (!dcheck(row[e] >= 0 && row[e] < c.page_size, c.err, kDbgGlobal)) continue;
            const size_t to = pg[e] * c.page_stride + ((size_t)h * c.page_size + row[e]) * c.d + part * 8;
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(c.k) + to) = kx[e];
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(c.v) + to) = vx[e];
        }
    }
    if (bad) atomicCAS(c.err, 0u, (unsigned)kErrPagedPage);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppend &pr, cudaStream_t stream) {
    PagedAppend a = pr;
    cudaError_t e = error_word_ptr(&a.c.err);
    if (e != cudaSuccess) return e;
    // one round of a block's threads, or several while that leaves enough blocks to
    // fill the GPU (blocks past a sequence's count end at once, but each costs a launch)
    const int round = kRowsAtOnce * kAppendThreads / (a.c.d / 8);
    const long long rows = (long long)a.c.B * a.c.Hkv;
    int sms = 0, stretch = round;
    if ((e = device_sms(&sms)) != cudaSuccess) return e;
    while (stretch < 4 * round && rows * ((a.n + 2LL * stretch - 1) / (2 * stretch)) >= 16LL * sms) stretch *= 2;
    const int stretches = a.n > stretch ? (a.n + stretch - 1) / stretch : 1;
    const long long blocks = rows * stretches;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    paged_append<<<(unsigned)blocks, kAppendThreads, 0, stream>>>(a, stretch, stretches);
    return cudaGetLastError();
}

}  // namespace lssar
