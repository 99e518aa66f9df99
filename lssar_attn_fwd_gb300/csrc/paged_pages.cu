// Paged cache, pages: taken from a list of free pages for new tokens, and given back.
//
// Sequence b holds ceil(lens[b] / page_size) pages.  Its needs (or what it gives back) are
// added up over the sequences before it, e_b, which says where in the list its pages
// lie: the list's end for reserve (entry free - 1 - k for the k-th page taken), behind it
// for release.  Each CTA takes a run of sequences: it adds up all lengths (8 bytes a
// sequence, from L2), scans its own run, and its warps copy the page numbers.  A launch's
// latency bounds it: reserving for 256 sequences takes 3.8 us of device time, releasing 96
// sequences of 32K tokens (400 KB of page numbers) 4.1, where the host's call takes 12 to 17.
#include "paged.cuh"
#include "tc_host.cuh"

namespace lssar {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Pages that sequence b takes or gives back: `count` from column `first` of its row on.
struct Change {
    int first, count;
    bool bad;
};

template <bool RESERVE>
__device__ __forceinline__ Change change_of(const PagedPages &a, int b) {
    const int cap = a.max_pages * a.page_size, len = a.lens[b];
    const int x = RESERVE && !a.other ? 1 : a.other[b];
    Change c;
    c.bad = len < 0 || len > cap || x < 0 || (RESERVE ? (long long)len + x > cap : x > len);
    const int up = a.page_size - 1;
    const int have = c.bad ? 0 : (len + up) / a.page_size, next = c.bad ? 0 : ((RESERVE ? len + x : x) + up) / a.page_size;
    c.first = RESERVE ? have : next;
    c.count = RESERVE ? next - have : have - next;
    return c;
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ long long block_sum(long long x, long long *part) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    long long s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w];
    return s;
}

template <bool RESERVE>
__global__ void __launch_bounds__(kThreads) paged_pages(const __grid_constant__ PagedPages a, int run) {
    __shared__ long long part[kWarps];
    __shared__ long long from[kThreads];   // of each sequence of a round: its first page's place
    __shared__ int first[kThreads], count[kThreads];
    const int tid = threadIdx.x, b0 = blockIdx.x * run, b1 = min(b0 + run, a.B);
    const int free_pages = *a.free_count;
    const bool usable = free_pages >= 0 && free_pages <= a.n_pages;
    bool bad_length = !usable, bad_page = false;
    // what the sequences before this run change, and those of all
    long long before = 0, all = 0;
    for (int b = tid; b < (RESERVE ? b0 : a.B); b += kThreads) {
        const Change c = change_of<RESERVE>(a, b);
        if (b < b0) before += c.count;
        all += c.count;
    }
    before = block_sum(before, part);
    if (!RESERVE) {
        all = block_sum(all, part);
        if (usable && free_pages + all > a.n_pages) bad_length = true;
    }
    const bool active = RESERVE ? usable : !bad_length;
    long long end = before;                // of the sequences up to here
#pragma unroll 1
    for (int base = b0; base < b1; base += kThreads) {
        const int b = base + tid;
        const bool mine = b < b1;
        Change c = {0, 0, false};
        if (mine) c = change_of<RESERVE>(a, b);
        bad_length |= c.bad;
        long long incl = c.count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if ((tid & 31) >= o) incl += y;
        }
        __syncthreads();
        if ((tid & 31) == 31) part[tid >> 5] = incl;
        __syncthreads();
        long long round = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < (tid >> 5)) incl += part[w];
            round += part[w];
        }
        incl += end;
        const bool served = active && !c.bad && (!RESERVE || c.count == 0 || incl <= free_pages);
        if (RESERVE && mine) a.counts_out[b] = served ? (a.other ? a.other[b] : 1) : 0;
        from[tid] = incl - c.count;
        first[tid] = c.first;
        count[tid] = served ? c.count : 0;
        __syncthreads();
        // threads for a sequence: a warp, or, where the run has fewer sequences than there are warps, more
        // (96 sequences of 2048 pages: 12.3 -> 4.1 us)
        const int here = min(kThreads, b1 - base), team = here >= kWarps ? 32 : kThreads >> (32 - __clz(here - 1));
        for (int i = tid / team; i < here; i += kThreads / team) {
            int *row = a.table + (size_t)(base + i) * a.max_pages + first[i];
#pragma unroll 4
            for (int j = tid % team; j < count[i]; j += team) {
                const long long k = from[i] + j;
                if (RESERVE) {
                    const int page = a.free_pages[free_pages - 1 - k];
                    const bool ok = (unsigned)page < (unsigned)a.n_pages;
                    bad_page |= !ok;
                    row[j] = ok ? page : -1;
                } else {
                    const int page = row[j];
                    bad_page |= (unsigned)page >= (unsigned)a.n_pages;
                    a.free_pages[free_pages + k] = page;
                }
            }
        }
        // the free pages left: all that fit, which end in one block's run
        if (RESERVE && usable) {
            const long long top = mine && incl <= free_pages ? incl : 0;
            long long most = top;
#pragma unroll
            for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
            __syncthreads();
            if ((tid & 31) == 0) part[tid >> 5] = most;
            __syncthreads();
            if (tid == 0 && end <= free_pages && (end + round > free_pages || (b1 == a.B && base + kThreads >= b1))) {
                long long taken = end;
                for (int w = 0; w < kWarps; ++w) taken = max(taken, part[w]);
                *a.free_out = (int)(free_pages - taken);
            }
            __syncthreads();
        }
        end += round;
    }
    if (tid == 0 && b1 == a.B) {
        if (!RESERVE) *a.free_out = active ? (int)(free_pages + all) : free_pages;
        else if (!usable) *a.free_out = free_pages;
    }
    if (bad_length) atomicCAS(a.err, 0u, (unsigned)kErrPagedLength);
    if (bad_page) atomicCAS(a.err, 0u, (unsigned)kErrPagedPage);
}

template <bool RESERVE>
cudaError_t launch(const PagedPages &pr, cudaStream_t stream) {
    PagedPages a = pr;
    cudaError_t e = error_word_ptr(&a.err);
    if (e != cudaSuccess) return e;
    int sms = 0;
    if ((e = device_sms(&sms)) != cudaSuccess) return e;
    const int run = (a.B + 2 * sms - 1) / (2 * sms);
    paged_pages<RESERVE><<<(a.B + run - 1) / run, kThreads, 0, stream>>>(a, run);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_reserve(const PagedPages &pr, cudaStream_t stream) { return launch<true>(pr, stream); }
cudaError_t launch_paged_release(const PagedPages &pr, cudaStream_t stream) { return launch<false>(pr, stream); }

}  // namespace lssar
