// Paged cache, eviction by added-up attention weight.
//
// Of the n = lens[b] cached tokens of a (sequence, key head), the `keep` of
// the highest rank stay: the protected ones (position < sinks, or position >
// newest - recent), then by score, equal scores by the lower slot.  Attention
// is a sum over a set, so the order of the slots carries nothing (a token's
// position is kept beside it), and the compaction moves as few rows as an
// in-place one can: the kept slots >= keep ("movers") go into the evicted
// slots < keep ("holes"), the j-th into the j-th.  No slot is both a source
// and a destination, so all moves are independent.
//
// Rank as a 32-bit key: a float's bits in the order of the values (-0 as +0),
// NaN below every number, all ones for a protected token.  One CTA per row
// finds the keep-th largest key by its four bytes from the highest down (a
// 256-bin histogram each), then walks the slots once in order, numbers the
// holes and the movers and lists them; a second kernel moves the rows.
#include <climits>

#include "paged.cuh"
#include "tc_host.cuh"

namespace lssar {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;

// Key of one slot (see above).
__device__ __forceinline__ unsigned rank_key(float s, int pos, int newest, int recent, int sinks) {
    // 64 bits: newest - recent may lie below the least int
    if (pos < sinks || (long long)pos > (long long)newest - recent) return 0xffffffffu;
    if (isnan(s)) return 0u;
    const unsigned u = __float_as_uint(s == 0.f ? 0.f : s);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of x over the block; *total = the block's sum.
__device__ int block_scan(int x, int *red, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = s;
    __syncthreads();
    int before = 0, sum = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
        if (w < warp) before += red[w];
        sum += red[w];
    }
    *total = sum;
    return before + s - x;
}

// src / dst: [B * Hkv][keep] lists, count: [B * Hkv].
__global__ void __launch_bounds__(kSelThreads) paged_select(const PagedEvict a, int *__restrict__ src, int *__restrict__ dst, int *__restrict__ count) {
    const PagedCache &c = a.c;
    __shared__ int red[kSelThreads / 32];
    __shared__ unsigned hist[256];
    __shared__ unsigned s_prefix, s_need;
    const int bh = blockIdx.x, b = bh / c.Hkv;
    const int n = paged_len(c, b);
    const size_t base = (size_t)bh * c.capacity();
    const float *sc = a.scores + base;
    const int *pos = a.positions + base;
    float *sc_out = a.scores_out + base;
    int *pos_out = a.positions_out + base;
    const bool in_place = a.scores == a.scores_out;
    // (a length outside the cache stays as it is, and nothing of its rows moves)
    if (bh % c.Hkv == 0 && threadIdx.x == 0) a.lens_out[b] = c.lens[b] == n ? min(n, a.keep) : c.lens[b];
    if (n <= a.keep) {
        if (threadIdx.x == 0) count[bh] = 0;
        for (int j = threadIdx.x; j < n; j += kSelThreads) {
            sc_out[j] = sc[j];
            pos_out[j] = pos[j];
        }
        return;
    }
    int newest = INT_MIN;
    for (int j = threadIdx.x; j < n; j += kSelThreads) newest = max(newest, pos[j]);
    newest = __reduce_max_sync(0xffffffffu, newest);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = newest;
    __syncthreads();
    for (int w = 0; w < kSelThreads / 32; ++w) newest = max(newest, red[w]);
    // the keep-th largest key, byte by byte; need: how many keys equal to it stay
    unsigned prefix = 0, need = a.keep;
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kSelThreads) {
            const unsigned key = rank_key(sc[j], pos[j], newest, a.recent, a.sinks);
            if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int bin = 255;
            unsigned left = need;
            while (hist[bin] < left) left -= hist[bin--];
            s_prefix = prefix | ((unsigned)bin << shift);
            s_need = left;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
    }
    // walk the slots in order
    int eq_before = 0, holes = 0, movers = 0;
    for (int j0 = 0; j0 < n; j0 += kSelThreads) {
        const int j = j0 + threadIdx.x;
        const float s = j < n ? sc[j] : 0.f;
        const int ps = j < n ? pos[j] : 0;
        const unsigned key = j < n ? rank_key(s, ps, newest, a.recent, a.sinks) : 0u;
        int total;
        const int eq = j < n && key == prefix;
        const int rank = eq_before + block_scan(eq, red, &total);
        eq_before += total;
        const bool kept = j < n && (key > prefix || (eq && rank < (int)need));
        const int hole = j < a.keep && !kept, mover = j >= a.keep && kept;
        const int at = block_scan(hole, red, &total);
        if (hole) dst[(size_t)bh * a.keep + holes + at] = j;
        holes += total;
        const int mat = block_scan(mover, red, &total);
        if (mover) src[(size_t)bh * a.keep + movers + mat] = j;
        movers += total;
        if (!in_place && j < a.keep && kept) {
            sc_out[j] = s;
            pos_out[j] = ps;
        }
    }
    if (threadIdx.x == 0) count[bh] = movers;
}

__global__ void __launch_bounds__(kMoveThreads) paged_move(const PagedEvict a, const int *__restrict__ src, const int *__restrict__ dst, const int *__restrict__ count) {
    const PagedCache &c = a.c;
    const int bh = blockIdx.x, b = bh / c.Hkv, h = bh % c.Hkv, parts = c.d / 8;
    const int part = threadIdx.x % parts, per = kMoveThreads / parts, n = count[bh];
    const size_t base = (size_t)bh * c.capacity();
    for (int i = blockIdx.y * per + threadIdx.x / parts; i < n; i += gridDim.y * per) {
        const int from = src[(size_t)bh * a.keep + i], to = dst[(size_t)bh * a.keep + i];
        if (part == 0) {
            a.scores_out[base + to] = a.scores[base + from];
            a.positions_out[base + to] = a.positions[base + from];
        }
        const int pf = paged_page(c, b, from / c.page_size), pt = paged_page(c, b, to / c.page_size);
        if (pf < 0 || pt < 0) continue;
        const size_t of = pf * c.page_stride + ((size_t)h * c.page_size + from % c.page_size) * c.d + part * 8;
        const size_t ot = pt * c.page_stride + ((size_t)h * c.page_size + to % c.page_size) * c.d + part * 8;
        auto *k = static_cast<uint16_t *>(c.k), *v = static_cast<uint16_t *>(c.v);
        const uint4 kx = *reinterpret_cast<const uint4 *>(k + of), vx = *reinterpret_cast<const uint4 *>(v + of);
        *reinterpret_cast<uint4 *>(k + ot) = kx;
        *reinterpret_cast<uint4 *>(v + ot) = vx;
    }
}

}  // namespace

size_t paged_evict_workspace_bytes(const PagedEvict &pr) {
    const size_t rows = (size_t)pr.c.B * pr.c.Hkv;
    return rows * pr.keep * 8 + rows * 4;
}

cudaError_t launch_paged_evict(const PagedEvict &pr, void *ws, cudaStream_t stream) {
    PagedEvict a = pr;
    cudaError_t e = error_word_ptr(&a.c.err);
    if (e != cudaSuccess) return e;
    const int rows = a.c.B * a.c.Hkv;
    int *src = static_cast<int *>(ws), *dst = src + (size_t)rows * a.keep, *count = dst + (size_t)rows * a.keep;
    paged_select<<<rows, kSelThreads, 0, stream>>>(a, src, dst, count);
    paged_move<<<dim3(rows, 16), kMoveThreads, 0, stream>>>(a, src, dst, count);
    return cudaGetLastError();
}

}  // namespace lssar
