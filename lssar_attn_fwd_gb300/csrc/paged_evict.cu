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
// NaN below every number, all ones for a protected token.
//
// paged_select: one thread-block cluster per row.  Each CTA takes an equal run of
// the row's slots and keeps their keys in shared memory, so that scores are read
// once and positions twice.  The keep-th largest key is found by its four bytes
// from the highest down: 256-bin histograms whose sums over the cluster meet
// in distributed shared memory.  Then each warp
// walks its own stretch of slots, ballots and sums over the block and the cluster
// number the holes and the movers, and their lists go to scratch.
// paged_move: all SMs move the rows, 16 bytes a lane, two rows of a group of
// threads at once.  (Moved by the selecting clusters, which leave SMs idle and
// have few loads in flight, 32 rows of 128K tokens took 226 us.)
//
// Long rows: HBM bounds the moves (8 bytes of each slot, 8d of each moved row), after a
// selection of a third to half of the time that overlaps nothing.  Short ones: latency; a row
// of one CTA goes through up to 24 block barriers with a few steps in shared memory between
// them, and the moves are a launch of their own (alone 16 and 8 us).
// Measured: 96 rows of 2K tokens 18.5 us, 96 rows of 16K tokens 66 us, 32 rows of 128K
// tokens 214-218 us; the moves of the last at 5.8 TB/s, rows of 256 bytes at scattered places.
#include <climits>
#include <cstdlib>

#include "paged.cuh"
#include "tc_host.cuh"
#include "tc_ptx.cuh"

namespace lssar {
namespace {

constexpr int kThreads = 512;
constexpr int kMoveThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;            // portable cluster size
constexpr int kCachedKeys = 18432;        // keys per CTA held in shared memory: two CTAs per SM (three up to about 18100)
constexpr int kChunk = 4096;              // slots per CTA that are worth another CTA
constexpr int kMoves = 2;                 // rows that a group of threads moves at once

constexpr unsigned kZeroKey = 0x80000000u;   // of a score 0

// Key of a score (see above), and whether its token is protected.
__device__ __forceinline__ unsigned score_key(float s) {
    if (isnan(s)) return 0u;
    const unsigned u = __float_as_uint(s == 0.f ? 0.f : s);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ bool is_protected(int pos, int newest, int recent, int sinks) {
    // 64 bits: newest - recent may lie below the least int
    return pos < sinks || (long long)pos > (long long)newest - recent;
}

// Shared memory that the cluster's other CTAs read.
struct Shared {
    int newest;
    unsigned hist[4][256];
    int holes, movers;
};

__device__ __forceinline__ int ld_cluster(const void *p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ptx::cluster_map(ptx::smem_u32(p), (uint32_t)rank)) : "memory");
    return v;
}

__device__ __forceinline__ unsigned dynamic_shared_bytes() {
    unsigned x;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(x));
    return x;
}

// Barrier of the row's CTAs.
__device__ __forceinline__ void row_sync(int ctas) {
    if (ctas == 1) __syncthreads();
    else ptx::cluster_sync();
}

// Exclusive prefix sums of x and y over the block, in thread order; *tx, *ty: the block's sums.
__device__ void block_scan(int &x, int &y, int2 *red, int *tx, int *ty) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int a = x, b = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, a, o), v = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += u;
            b += v;
        }
    }
    __syncthreads();
    if (lane == 31) red[warp] = make_int2(a, b);
    __syncthreads();
    int2 w = lane < kWarps ? red[lane] : make_int2(0, 0);
    int2 s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s.x, o), v = __shfl_up_sync(0xffffffffu, s.y, o);
        if (lane >= o) {
            s.x += u;
            s.y += v;
        }
    }
    *tx = __shfl_sync(0xffffffffu, s.x, 31);
    *ty = __shfl_sync(0xffffffffu, s.y, 31);
    x = a - x + __shfl_sync(0xffffffffu, s.x - w.x, warp);
    y = b - y + __shfl_sync(0xffffffffu, s.y - w.y, warp);
}

// src / dst: [B * Hkv][keep] slots of the movers and the holes.  CACHED: the
// run's keys are in shared memory; else each pass makes them again.
template <bool CACHED>
__global__ void __launch_bounds__(kThreads, 3)
paged_select(const __grid_constant__ PagedEvict a, int *__restrict__ src, int *__restrict__ dst, int *__restrict__ count, int ctas) {
    ptx::launch_dependents();
    const PagedCache &c = a.c;
    extern __shared__ unsigned cached[];
    __shared__ Shared sh;
    __shared__ int2 red[kWarps];
    __shared__ unsigned s_bin, s_left;
    __shared__ bool s_all;
    const int bh = blockIdx.x / ctas, rank = blockIdx.x % ctas, b = bh / c.Hkv, h = bh % c.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = paged_len(c, b);
    const size_t base = (size_t)bh * c.capacity();
    const float *sc = a.scores + base;
    const int *pos = a.positions + base;
    float *sc_out = a.scores_out + base;
    int *pos_out = a.positions_out + base;
    // (a length outside the cache stays as it is, and nothing of its rows moves)
    if (h == 0 && rank == 0 && threadIdx.x == 0) a.lens_out[b] = c.lens[b] == n ? min(n, a.keep) : c.lens[b];
    // slots [lo, hi) are this CTA's
    const int run = ((n + ctas - 1) / ctas + 3) & ~3, lo = min(n, rank * run), hi = min(n, lo + run);
    if (a.scores != a.scores_out)   // the holes' values follow below
#pragma unroll 4
        for (int j = lo + threadIdx.x; j < min(hi, a.keep); j += kThreads) {
            sc_out[j] = sc[j];
            pos_out[j] = pos[j];
        }
    // (one answer for the whole cluster; in the debug build a run that its shared memory does not hold)
    if (n <= a.keep || !dcheck(b < c.B && (!CACHED || (unsigned)run * 4u <= dynamic_shared_bytes()), c.err, kDbgItem)) {
        if (rank == 0 && threadIdx.x == 0) count[bh] = 0;
        return;
    }
    // the newest position of the row; the scores' keys
    int newest = INT_MIN;
#pragma unroll 8
    for (int j = lo + threadIdx.x; j < hi; j += kThreads) {
        newest = max(newest, pos[j]);
        if (CACHED) cached[j - lo] = score_key(sc[j]);
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) red[warp].x = newest;
    for (int i = threadIdx.x; i < 4 * 256; i += kThreads) reinterpret_cast<unsigned *>(sh.hist)[i] = 0;
    __syncthreads();
    if (warp == 0) {
        newest = __reduce_max_sync(0xffffffffu, lane < kWarps ? red[lane].x : INT_MIN);
        if (lane == 0) sh.newest = newest;
    }
    row_sync(ctas);
    newest = __reduce_max_sync(0xffffffffu, lane < ctas ? ld_cluster(&sh.newest, lane) : INT_MIN);
    if (CACHED) {
#pragma unroll 8
        for (int j = lo + threadIdx.x; j < hi; j += kThreads)
            if (is_protected(pos[j], newest, a.recent, a.sinks)) cached[j - lo] = 0xffffffffu;
    }
    auto key_of = [&](int j) {
        if (CACHED) return cached[j - lo];
        return is_protected(pos[j], newest, a.recent, a.sinks) ? 0xffffffffu : score_key(sc[j]);
    };
    // the keep-th largest key, byte by byte; left: how many of the keys with its
    // leading bytes are among the highest `keep`
    unsigned prefix = 0, left = a.keep;
    const int steps = (hi - lo + kThreads - 1) / kThreads;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        unsigned zeros = 0, safes = 0;
#pragma unroll 2
        for (int i = 0; i < steps; ++i) {   // (a thread meets the keys that it made)
            const int j = lo + i * kThreads + threadIdx.x;
            const unsigned key = j < hi ? key_of(j) : 0u;
            const bool in = j < hi && (pass == 0 || (key >> (shift + 8)) == (prefix >> (shift + 8)));
            // counted apart: many tokens have no weight at all, and protected ones come
            // together (lanes with equal bins found by a match cost more than they saved)
            const bool zero = key == kZeroKey, safe = key == 0xffffffffu;
            zeros += in && zero;
            safes += in && safe;
            if (in && !zero && !safe) atomicAdd(&sh.hist[pass][(key >> shift) & 255u], 1u);
        }
        zeros = __reduce_add_sync(0xffffffffu, zeros);
        safes = __reduce_add_sync(0xffffffffu, safes);
        if (lane == 0) {
            if (zeros) atomicAdd(&sh.hist[pass][(kZeroKey >> shift) & 255u], zeros);
            if (safes) atomicAdd(&sh.hist[pass][255], safes);
        }
        row_sync(ctas);
        // sums over the cluster, then from the highest bin down: thread t has bin 255 - t
        int cnt = 0, zero = 0, t0, t1;
        if (threadIdx.x < 256)
#pragma unroll 1
            for (int r = 0; r < ctas; r += 2) {   // (a cluster of one reads itself)
                const int x = ld_cluster(&sh.hist[pass][255 - threadIdx.x], r), y = r + 1 < ctas ? ld_cluster(&sh.hist[pass][255 - threadIdx.x], r + 1) : 0;
                cnt += x + y;
            }
        int above = cnt;
        block_scan(above, zero, red, &t0, &t1);
        if (threadIdx.x < 256 && above < (int)left && above + cnt >= (int)left) {
            s_bin = 255 - threadIdx.x;
            s_left = left - above;
            s_all = above + cnt == (int)left;
        }
        __syncthreads();
        prefix |= s_bin << shift;
        left = s_left;
        if (s_all) {   // the whole bin stays: every key from its least on, and none is equal to `prefix`
            prefix -= 1;
            left = 0;
            break;
        }
    }
    // of the keys equal to `prefix` the first `left` stay: those of the CTAs
    // before this one are in the last histogram
    int eq_before = 0;
    if (left)
#pragma unroll 1
        for (int r = 0; r < rank; ++r) eq_before += ld_cluster(&sh.hist[3][prefix & 255u], r);
    // each warp walks its own stretch of slots in order, 32 at a time; ballots rank
    // the slots within it
    const int stretch = (((hi - lo + kWarps - 1) / kWarps) + 31) & ~31;
    const int w0 = min(hi, lo + warp * stretch), w1 = min(hi, w0 + stretch);
    const unsigned below = (1u << lane) - 1;
    int eq = 0;
    if (left)
#pragma unroll 2
        for (int j = w0 + lane; j - lane < w1; j += 32) eq += __popc(__ballot_sync(0xffffffffu, j < w1 && key_of(j) == prefix));
    __syncthreads();
    if (lane == 0) red[warp] = make_int2(eq, 0);
    __syncthreads();
    int rank0 = eq_before + __reduce_add_sync(0xffffffffu, lane < warp ? red[lane].x : 0);
    // whether slot j (of this lane) stays; counts the keys equal to `prefix` as it goes
    auto stays = [&](int j, int &seen) {
        const unsigned key = j < w1 ? key_of(j) : 0u;
        const bool same = j < w1 && key == prefix;
        const unsigned all = __ballot_sync(0xffffffffu, same);
        const bool s = j < w1 && (key > prefix || (same && seen + __popc(all & below) < (int)left));
        seen += __popc(all);
        return s;
    };
    int holes = 0, movers = 0, seen = rank0;
#pragma unroll 2
    for (int j = w0 + lane; j - lane < w1; j += 32) {
        const bool s = stays(j, seen);
        holes += __popc(__ballot_sync(0xffffffffu, j < w1 && j < a.keep && !s));
        movers += __popc(__ballot_sync(0xffffffffu, j >= a.keep && s));
    }
    __syncthreads();
    if (lane == 0) red[warp] = make_int2(holes, movers);
    __syncthreads();
    holes = __reduce_add_sync(0xffffffffu, lane < warp ? red[lane].x : 0);
    movers = __reduce_add_sync(0xffffffffu, lane < warp ? red[lane].y : 0);
    if (warp == 0) {
        const int x = __reduce_add_sync(0xffffffffu, lane < kWarps ? red[lane].x : 0), y = __reduce_add_sync(0xffffffffu, lane < kWarps ? red[lane].y : 0);
        if (lane == 0) {
            sh.holes = x;
            sh.movers = y;
        }
    }
    row_sync(ctas);
    int total = 0;
#pragma unroll 1
    for (int r = 0; r < ctas; ++r) {
        const int x = ld_cluster(&sh.holes, r), y = ld_cluster(&sh.movers, r);
        if (r < rank) {
            holes += x;
            movers += y;
        }
        total += x;
    }
    int *to_list = dst + (size_t)bh * a.keep, *from_list = src + (size_t)bh * a.keep;
    seen = rank0;
#pragma unroll 2
    for (int j = w0 + lane; j - lane < w1; j += 32) {
        const bool s = stays(j, seen), hole = j < w1 && j < a.keep && !s, mover = j >= a.keep && s;
        const unsigned hm = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
        const int hi_at = holes + __popc(hm & below), mo_at = movers + __popc(mm & below);
        if (hole && dcheck(hi_at < a.keep, c.err, kDbgGlobal)) to_list[hi_at] = j;
        if (mover && dcheck(mo_at < a.keep, c.err, kDbgGlobal)) from_list[mo_at] = j;
        holes += __popc(hm);
        movers += __popc(mm);
    }
    if (rank == 0 && threadIdx.x == 0) count[bh] = total;
    row_sync(ctas);   // no CTA's shared memory is read after this
}

// Moves the rows of the lists: `splits` blocks per (sequence, key head).
__global__ void __launch_bounds__(kMoveThreads, 4) paged_move(const __grid_constant__ PagedEvict a, const int *__restrict__ src, const int *__restrict__ dst, const int *__restrict__ count, int splits) {
    const PagedCache &c = a.c;
    const int bh = blockIdx.x / splits, rank = blockIdx.x - bh * splits, b = bh / c.Hkv, h = bh - b * c.Hkv;
    const int *from_list = src + (size_t)bh * a.keep, *to_list = dst + (size_t)bh * a.keep;
    const size_t base = (size_t)bh * c.capacity();
    const float *sc = a.scores + base;
    const int *pos = a.positions + base;
    float *sc_out = a.scores_out + base;
    int *pos_out = a.positions_out + base;
    ptx::grid_dependency_wait();
    int total = __ldcg(count + bh);
    if (!dcheck(total >= 0 && total <= a.keep, c.err, kDbgItem)) total = 0;
    // scores and positions, a thread each
    for (int i = rank * kMoveThreads + threadIdx.x; i < total; i += splits * kMoveThreads) {
        const int from = __ldcg(from_list + i), to = __ldcg(to_list + i);
        if (!dcheck(from >= a.keep && from < c.capacity() && to >= 0 && to < a.keep, c.err, kDbgGlobal)) continue;
        sc_out[to] = sc[from];
        pos_out[to] = pos[from];
    }
    // d / 8 threads per row, kMoves rows of a group at once: the places, the pages, then
    // the rows' loads are in flight together
    const int parts = c.d / 8, part = threadIdx.x % parts, groups = splits * (kMoveThreads / parts);
    auto *k = static_cast<uint16_t *>(c.k), *v = static_cast<uint16_t *>(c.v);
    const int *table = c.table + (size_t)b * c.max_pages;
    bool bad = false;
#pragma unroll 1
    for (int i0 = rank * (kMoveThreads / parts) + threadIdx.x / parts; i0 < total; i0 += kMoves * groups) {
        int from[kMoves], to[kMoves];
#pragma unroll
        for (int e = 0; e < kMoves; ++e) {
            const int i = i0 + e * groups;
            from[e] = i < total ? __ldcg(from_list + i) : -1;
            to[e] = i < total ? __ldcg(to_list + i) : 0;
            if (!dcheck(from[e] < c.capacity() && to[e] >= 0 && to[e] < a.keep, c.err, kDbgGlobal)) from[e] = -1, to[e] = 0;
        }
        int pf[kMoves], pt[kMoves], fr[kMoves], tr[kMoves];
#pragma unroll
        for (int e = 0; e < kMoves; ++e) {
            const int fi = max(from[e], 0) / c.page_size, ti = to[e] / c.page_size;
            fr[e] = from[e] - fi * c.page_size;
            tr[e] = to[e] - ti * c.page_size;
            pf[e] = table[fi];
            pt[e] = table[ti];
        }
        long long of[kMoves], ot[kMoves];
#pragma unroll
        for (int e = 0; e < kMoves; ++e) {
            const bool page = (unsigned)pf[e] < (unsigned)c.n_pages && (unsigned)pt[e] < (unsigned)c.n_pages;
            of[e] = from[e] >= 0 && page ? pf[e] * c.page_stride + ((long long)h * c.page_size + fr[e]) * c.d + part * 8 : -1;
            ot[e] = pt[e] * c.page_stride + ((long long)h * c.page_size + tr[e]) * c.d + part * 8;
            bad |= from[e] >= 0 && !page;
        }
        uint4 kx[kMoves], vx[kMoves];
#pragma unroll
        for (int e = 0; e < kMoves; ++e)
            if (of[e] >= 0) {
                kx[e] = *reinterpret_cast<const uint4 *>(k + of[e]);
                vx[e] = *reinterpret_cast<const uint4 *>(v + of[e]);
            }
#pragma unroll
        for (int e = 0; e < kMoves; ++e)
            if (of[e] >= 0) {
                *reinterpret_cast<uint4 *>(k + ot[e]) = kx[e];
                *reinterpret_cast<uint4 *>(v + ot[e]) = vx[e];
            }
    }
    if (bad) atomicCAS(c.err, 0u, (unsigned)kErrPagedPage);
}

template <bool CACHED>
cudaError_t launch_select(const PagedEvict &a, int *src, int *dst, int *count, int ctas, int run, cudaStream_t stream) {
    const int rows = a.c.B * a.c.Hkv, smem = CACHED ? run * 4 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static PerDeviceOnce once;
    const cudaError_t e = per_device_once(once, nullptr, [](int &) {
        return cudaFuncSetAttribute(paged_select<CACHED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCachedKeys * 4);
    });
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, paged_select<CACHED>, a, src, dst, count, ctas);
}

}  // namespace

size_t paged_evict_workspace_bytes(const PagedEvict &pr) { return (size_t)pr.c.B * pr.c.Hkv * (pr.keep * 8 + 4); }

cudaError_t launch_paged_evict(const PagedEvict &pr, void *ws, cudaStream_t stream) {
    PagedEvict a = pr;
    cudaError_t e = error_word_ptr(&a.c.err);
    if (e != cudaSuccess) return e;
    int *src = static_cast<int *>(ws), *dst = src + (size_t)a.c.B * a.c.Hkv * a.keep, *count = dst + (size_t)a.c.B * a.c.Hkv * a.keep;
    // CTAs per row by the longest row that the table has room for, in one wave of three
    // per SM (96 rows of 16K tokens: 2, 4 and 8 CTAs each took 77, 68 and 82 us; a run halved
    // for the wave's sake is at most kCachedKeys / 2, of which three do fit an SM), or
    // more while the keys do not fit shared memory
    const int cap = a.c.capacity();
    const long long rows = (long long)a.c.B * a.c.Hkv;
    int sms = 0, ctas = 1;
    if ((e = device_sms(&sms)) != cudaSuccess) return e;
    while (ctas < kMaxCluster && cap > ctas * kChunk && (2 * ctas * rows <= 3 * sms || cap > ctas * kCachedKeys)) ctas *= 2;
    const int run = ((cap + ctas - 1) / ctas + 3) & ~3;
    e = run <= kCachedKeys ? launch_select<true>(a, src, dst, count, ctas, run, stream) : launch_select<false>(a, src, dst, count, ctas, run, stream);
    if (e != cudaSuccess) return e;
    // two waves of four blocks per SM, more where there are more rows, but not more
    // than the moves of a full row give work to
    const int at_once = kMoves * kMoveThreads / (a.c.d / 8), most = (a.keep + at_once - 1) / at_once;
    long long splits = (8LL * sms + rows - 1) / rows;
    if (splits > most) splits = most;
    if (rows * splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * splits));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_move, a, (const int *)src, (const int *)dst, (const int *)count, (int)splits);
}

}  // namespace lssar
