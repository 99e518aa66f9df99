// Paged cache, decode: one new query row per head against a sequence's pages,
// in every mode of the forward (row i = the sequence's length), grouped heads,
// and the attention weight that each cached token receives added up.
//
// Mathematics, per (sequence b, query head): z_j = the score in log2 units,
// phi_j = the mode's normaliser, S1 = sum phi_j, m = max z_j; the weights are
// w_j = phi_j (softmax: 2^(z_j - m)), or with re-weighting max(kappa phi_j +
// beta, 0)^p with kappa, beta from S1, m and i; out = sum w_j v_j / sum w_j.
//
// What bounds it: every key and value row is read once from HBM, 4d bytes per
// (token, key head) against 4Gd flops for a group of G query heads.
//
// Split.  The tokens of all sequences are cut into tiles of 64 keys of one key
// head, numbered through (sequence, key head, block of 8 query heads, tile); each
// CTA takes an equal run of tiles wherever rows begin or end, so that lengths
// of any mix load the SMs evenly.  The part of a row inside one run is a segment.
// The lengths are on the device: each warp finds its run by a prefix sum.
//   softmax, LSSA: paged_stream<kBoth>   one pass over K and V tiles, weights
//                  relative to a running maximum (softmax);
//   re-weighting:  paged_stream<kScores> K tiles -> z (scratch), (m, S1) per segment,
//                  paged_stream<kValues> row constants from all of the row's
//                  segments, z -> w, V tiles (their copies start before the
//                  scores kernel ends);
//   then           paged_join            sums the segments of each row, and adds
//                  each token's normalised weights to its score.
// Each kernel is a programmatic dependent of the one before it.
//
// Products on mma.sync m16n8k16: a decode row has G <= 8 query heads per key head
// in a block, which a 128-row tcgen05 tile would leave almost empty, and the
// tensor work is a small part of the time that HBM needs.  The 16 rows of an
// operand carry the 8 heads and, for free, something else that is needed:
//   scores: rows 8-15 the queries, rows 0-7 the tile's own 8 keys, so that one
//           product gives q.k and, on the diagonal, |k|^2;
//   values: rows 8-15 the weights rounded to 16 bits, rows 0-7 what the rounding
//           left over, so that weights keep 16 bits (bf16) or more.
// K and V tiles come by TMA (128-byte swizzle) one page piece at a time.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "paged.cuh"
#include "row_weights.cuh"
#include "tc_host.cuh"
#include "tc_ptx.cuh"

namespace lssar {
namespace {

enum Phase : int { kScores = 0, kValues = 1, kBoth = 2 };

constexpr int kTile = 64;                     // keys per tile
constexpr int kWarps = 4;                     // compute warps, 16 keys of each tile each
constexpr int kCompute = kWarps * 32;
constexpr int kBlock = kCompute + 32;         // + the producer warp
constexpr int kHeads = 8;                     // query heads per block of heads
constexpr int kMaxGroup = 128;                // H / Hkv
constexpr float kLowest = -3.0e38f;           // below every score, and finite
constexpr uint64_t kWaitLimitNs = 2000000000ull;
enum : unsigned { kErrFull = 53, kErrEmpty, kErrDrain };

// Run of tiles of this CTA and the row constants of the split, known to every warp.
struct Split {
    int heads_rows;        // Hkv * blocks: rows per sequence
    int blocks;            // blocks of kHeads query heads per key head
    int zg;                // heads stored per tile: min(G, kHeads)
    int ctas;              // CTAs that share the tiles
    int min_run;           // tiles per CTA at least
};

struct Scratch {
    float *z;              // [tile][zg][kTile]
    float2 *stats;         // [segment][zg]: max of z, sum of phi
    float2 *sums;          // [segment][zg]: reference of the exponent (softmax), sum of w
    float *o;              // [segment][zg][D]: sum of w v
    float4 *rowc;          // [row][zg]: m, kappa, beta
};

struct Args {
    PagedDecode a;
    Split sp;
    Scratch s;
};

// A place in the numbering of the tiles.
struct Place {
    long long t;           // number of the tile
    int b, hr, tile;       // sequence, row of the sequence, tile of the row
    int n, nt;             // length and tiles of the sequence
};

__device__ __forceinline__ int tiles_of(const PagedCache &c, int b) { return (paged_len(c, b) + kTile - 1) / kTile; }

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Tiles of sequences [0, upto) for one row of each (the whole warp calls it).
__device__ long long tiles_before(const PagedCache &c, int upto) {
    long long x = 0;
    for (int b = threadIdx.x & 31; b < upto; b += 32) x += tiles_of(c, b);
    return warp_sum(x);
}

// Tiles per CTA: an equal share of the total.
__device__ __forceinline__ int run_length(const Split &sp, long long total) {
    const long long run = (total + sp.ctas - 1) / sp.ctas;
    return (int)(run < sp.min_run ? sp.min_run : run);
}

// The place of tile t < total (the whole warp calls it).
__device__ Place locate(const PagedCache &c, int rows_per_seq, long long t) {
    const int lane = threadIdx.x & 31;
    Place p;
    long long before = 0;
    for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < c.B ? paged_len(c, b) : 0, nt = (n + kTile - 1) / kTile;
        long long end = (long long)nt * rows_per_seq;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + end > t);
        if (hit) {
            const int l = __ffs(hit) - 1;
            p.n = __shfl_sync(0xffffffffu, n, l);
            p.nt = __shfl_sync(0xffffffffu, nt, l);
            const long long start = before + __shfl_sync(0xffffffffu, end, l) - (long long)p.nt * rows_per_seq;
            p.b = b0 + l;
            p.hr = (int)((t - start) / p.nt);
            p.tile = (int)((t - start) % p.nt);
            p.t = t;
            return p;
        }
        before += __shfl_sync(0xffffffffu, end, 31);
    }
}

// On to the first tile of the next row that has one.
__device__ __forceinline__ void next_row(const PagedCache &c, int rows_per_seq, Place &p) {
    p.tile = 0;
    if (++p.hr < rows_per_seq) return;
    p.hr = 0;
    do {
        if (++p.b >= c.B) return;
        p.n = paged_len(c, p.b);
        p.nt = (p.n + kTile - 1) / kTile;
    } while (p.nt == 0);
}

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return ptx::pack_bf16x2(lo, hi); }
    static __device__ __forceinline__ float2 unpack(uint32_t x) {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return ptx::pack_f16x2(lo, hi); }
    static __device__ __forceinline__ float2 unpack(uint32_t x) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    }
    static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Address of the 16-byte piece `chunk` of a tile's row: halves of 64 columns,
// each kTile rows of 128 bytes with TMA's 128-byte swizzle.
__device__ __forceinline__ uint32_t piece(uint32_t tile, int row, int chunk) {
    return tile + (chunk >> 3) * (kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory"); }

template <int D, int PHASE>
struct Config {
    static constexpr int kStageBytes = kTile * D * 2;
    static constexpr int kStages = D == 64 ? (PHASE == kScores ? 6 : 5) : (PHASE == kScores ? 4 : 3);
    static constexpr int kPerSm = D == 64 ? 4 : 3;
    static constexpr int kMerge = PHASE == kScores ? 0 : kWarps * kHeads * D * 4;   // bytes of the warps' value sums
};

struct Shared {
    uint64_t full[8], empty[8];
    int bad[8];                     // the stage's tile names a page that is none
    float2 red[kWarps][kHeads];
    float4 rowc[kHeads];
    int abort_flag;
};

__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, Shared *sh, unsigned *err, unsigned code, bool honour_abort) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t spin = 1;; ++spin) {
        if (ptx::mbar_try_wait_sleep(bar, parity, 200000)) return true;
        if ((spin & 15u) == 0) {
            if (honour_abort && *(volatile int *)&sh->abort_flag) return false;
            if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
                atomicCAS(err, 0u, code);
                *(volatile int *)&sh->abort_flag = 1;
                return false;
            }
        }
    }
}

// The segments of the row that starts at tile `start`: CTAs first..last, whose
// scratch entries are row + first .. row + last (both grow along the numbering,
// so that no two segments share one).
struct Segments {
    long long first, count;
};
__device__ __forceinline__ Segments segments_of(long long row, long long start, int nt, int run) {
    const long long a = start / run, b = (start + nt - 1) / run;
    return Segments{row + a, b - a + 1};
}

// (m, s) pairs of sums relative to 2^m.
__device__ __forceinline__ float2 join_pair(float2 x, float2 y) {
    // NaN (a row that must not be used) stays: fmaxf alone would drop it
    const float m = isnan(x.x) || isnan(y.x) ? NAN : fmaxf(x.x, y.x);
    return make_float2(m, x.y * ptx::ex2(x.x - m) + y.y * ptx::ex2(y.x - m));
}

// Row constants m, kappa, beta from the row's maximum and normaliser sum.
__device__ __forceinline__ float4 row_constants(int mode, int n, float m, float s1) {
    float kappa = 1.f, beta = 0.f;
    if (is_reweight(mode)) {
        const float theta = n <= 3 ? 0.f : s1 / (float)n, top = phi(mode, m, m), den = top - theta;
        if (den > 1e-5f * top + 2e-5f) {   // the prefill kernel's near-uniform band
            kappa = 1.f / den;
            beta = -theta * kappa;
        } else {
            kappa = 0.f;   // all-zero re-weighted row: uniform
            beta = 1.f;
        }
    }
    if (isnan(m) || isnan(s1)) kappa = NAN;
    return make_float4(m, kappa, beta, 0.f);
}

__device__ __forceinline__ float weight(int mode, int p, float z, const float4 &rc) {
    const float y = fmaf(phi(mode, z, rc.x), rc.y, rc.z);
    // max(y, 0) that keeps NaN
    return is_reweight(mode) ? powi(y < 0.f ? 0.f : y, p) : y;
}

// Producer warp: the tiles of the CTA's run, in order, through the ring.
template <int D, int PHASE>
__device__ void produce(const Args &g, const CUtensorMap *km, const CUtensorMap *vm, Shared *sh, uint32_t ring, Place p, long long t1, int piece_rows) {
    using C = Config<D, PHASE>;
    constexpr int kPer = PHASE == kBoth ? 2 : 1;   // stages per tile
    const PagedCache &c = g.a.c;
    const int lane = threadIdx.x & 31, pieces = kTile / piece_rows;
    // the page of this lane's piece of a tile; -1: past the row's end, -2: none of the pool
    auto look_up = [&](const Place &q) {
        const int s0 = q.tile * kTile + lane * piece_rows;
        if (lane >= pieces || s0 >= q.n) return -1;
        const int pg = paged_page(c, q.b, s0 / c.page_size);
        return pg < 0 ? -2 : pg;
    };
    int it = 0, pg = look_up(p);
    while (true) {
        Place q = p;
        ++q.t;
        int next = -1;
        if (q.t < t1) {
            if (++q.tile == q.nt) next_row(c, g.sp.heads_rows, q);
            next = look_up(q);
        }
        const unsigned ok = __ballot_sync(0xffffffffu, pg >= 0), bad = __ballot_sync(0xffffffffu, pg == -2);
        const int s0 = p.tile * kTile + lane * piece_rows;
        const int y = p.hr / g.sp.blocks * c.page_size + s0 % c.page_size;
        bool go = true;
#pragma unroll
        for (int u = 0; u < kPer; ++u, ++it) {
            const int s = it % C::kStages, use = it / C::kStages;
            if (use > 0) go = __all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh->empty[s]), (use - 1) & 1, sh, c.err, kErrEmpty, true));
            if (!go) break;
            const uint32_t full = ptx::smem_u32(&sh->full[s]), dst = ring + s * C::kStageBytes + lane * piece_rows * 128;
            const CUtensorMap *map = PHASE == kValues || u == 1 ? vm : km;
            if (lane == 0) {
                sh->bad[s] = bad != 0;
                ptx::mbar_arrive_expect_tx(full, (uint32_t)__popc(ok) * piece_rows * D * 2);
            }
            __syncwarp();
            if (pg >= 0 && dcheck(y >= 0 && y + piece_rows <= c.Hkv * c.page_size && pg < c.n_pages && lane < pieces, c.err, kDbgTma)) {
                ptx::tma_load_3d(dst, map, full, 0, y, pg);
                if (D == 128) ptx::tma_load_3d(dst + kTile * 128, map, full, 64, y, pg);
            }
        }
        if (!go || q.t >= t1) break;
        p = q;
        pg = next;
    }
    // the last copies have landed before the CTA ends
    if (lane == 0)
        for (int i = max(0, it - C::kStages); i < it; ++i)
            bounded_wait(ptx::smem_u32(&sh->full[i % C::kStages]), (i / C::kStages) & 1, sh, c.err, kErrDrain, false);
    __syncwarp();
}

// One segment's rows of 16 keys per warp: the scores z of the warp's 16 keys
// (two blocks of 8) for head lane / 4, keys 2 (lane % 4) + {0, 1} of each block.
template <typename T, int D>
__device__ __forceinline__ void score_tile(uint32_t tile, const uint32_t (&qf)[D / 16][2], float scale, bool raw, float2 (&z)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const int row = 16 * warp + 8 * u + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t r[4];
            ldsm4(r, piece(tile, row, 4 * kk + (lane >> 3)));
            Elem<T>::mma(d, r[0], qf[2 * kk][0], r[1], qf[2 * kk][1], r[0], r[1]);
            Elem<T>::mma(d, r[2], qf[2 * kk + 1][0], r[3], qf[2 * kk + 1][1], r[2], r[3]);
        }
        z[u] = make_float2(scale * d[2], scale * d[3]);
        if (!raw) {
            // |k|^2 of keys 2c and 2c + 1 is on the diagonal: rows 2c, 2c + 1 of the upper half
            const int c = lane & 3;
            const float ka = __shfl_sync(0xffffffffu, d[0], 9 * c), kb = __shfl_sync(0xffffffffu, d[1], 9 * c + 4);
            z[u].x *= rsqrtf(fmaxf(ka, 1e-24f));   // |k| clamped at 1e-12 as everywhere
            z[u].y *= rsqrtf(fmaxf(kb, 1e-24f));
        }
    }
}

// Adds w v of the warp's 16 keys to o (n8 blocks of columns; [0..1] from the
// weights' remainders, [2..3] from the rounded weights).
template <typename T, int D>
__device__ __forceinline__ void value_tile(uint32_t tile, const float2 (&w)[2], int left, float (&o)[D / 8][4]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        hi[u] = Elem<T>::pack(w[u].x, w[u].y);
        const float2 r = Elem<T>::unpack(hi[u]);
        lo[u] = Elem<T>::pack(w[u].x - r.x, w[u].y - r.y);
    }
    // rows at or past `left` of the tile hold anything (0 * NaN): clear them
    const bool tail = left < kTile;
    uint32_t mask[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int j = 16 * warp + 8 * u + 2 * c;
        mask[u] = (j < left ? 0xffffu : 0u) | (j + 1 < left ? 0xffff0000u : 0u);
    }
    const int row = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
    for (int np = 0; np < D / 16; ++np) {
        uint32_t r[4];
        ldsm4t(r, piece(tile, row, 2 * np + (lane >> 4)));
        if (tail) {
            r[0] &= mask[0];
            r[1] &= mask[1];
            r[2] &= mask[0];
            r[3] &= mask[1];
        }
        Elem<T>::mma(o[2 * np], lo[0], hi[0], lo[1], hi[1], r[0], r[1]);
        Elem<T>::mma(o[2 * np + 1], lo[0], hi[0], lo[1], hi[1], r[2], r[3]);
    }
}

template <typename T, int D, int PHASE>
__global__ void __launch_bounds__(kBlock, (Config<D, PHASE>::kPerSm))
paged_stream(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, const __grid_constant__ Args g, int piece_rows) {
    using C = Config<D, PHASE>;
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const PagedCache &c = g.a.c;
    const uint32_t ring = (ptx::smem_u32(dyn) + 1023u) & ~1023u;
    float *merge = reinterpret_cast<float *>(dyn + (ring - ptx::smem_u32(dyn)) + C::kStages * C::kStageBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int mode = g.a.mode, p_exp = g.a.p, G = g.a.H / c.Hkv;
    const bool raw = !uses_normalised_qk(mode);
    ptx::launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.empty[s]), kWarps);
        }
        sh.abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    const long long total = tiles_before(c, c.B) * g.sp.heads_rows;
    const int run = run_length(g.sp, total);
    const long long t0 = (long long)blockIdx.x * run, t1 = t0 + run < total ? t0 + run : total;
    __syncthreads();
    if (t0 >= total) {
        if (PHASE == kValues) ptx::grid_dependency_wait();   // this grid ends after the one before it
        return;
    }
    Place p = locate(c, g.sp.heads_rows, t0);
    if (warp == kWarps) {
        produce<D, PHASE>(g, &km, &vm, &sh, ring, p, t1, piece_rows);
        return;
    }
    if (PHASE == kValues) ptx::grid_dependency_wait();   // z and the segments' statistics
    const int head = lane >> 2, c4 = lane & 3;
    int it = 0;
    while (p.t < t1) {   // one segment per turn
        const long long row = (long long)p.b * g.sp.heads_rows + p.hr, start = p.t - p.tile, seg = row + blockIdx.x;
        const int g0 = p.hr % g.sp.blocks * kHeads, heads = min(kHeads, G - g0);
        const int cnt = (int)(t1 - p.t < p.nt - p.tile ? t1 - p.t : p.nt - p.tile);
        const bool mine = head < heads;
        // queries (rows past the block's heads are zero) and the row's factor
        uint32_t qf[D / 16][2];
        float scale = 0.f;
        if (PHASE != kValues) {
            const int hq = p.hr / g.sp.blocks * G + g0 + head;
            const uint16_t *q = static_cast<const uint16_t *>(g.a.q) + p.b * g.a.q_b + hq * g.a.q_h;
            float ss = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    qf[kk][u] = mine ? *reinterpret_cast<const uint32_t *>(q + 16 * kk + 8 * u + 2 * c4) : 0u;
                    const float2 x = Elem<T>::unpack(qf[kk][u]);
                    ss += x.x * x.x + x.y * x.y;
                }
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            const float log2e = 1.4426950408889634f;
            scale = raw ? log2e * rsqrtf((float)D) : log2e * logf((float)D) * logf((float)p.n) / fmaxf(sqrtf(ss), 1e-12f);
        }
        float4 rc = make_float4(0.f, 1.f, 0.f, 0.f);
        if (PHASE == kValues) {
            // the row's constants: 16 threads per head over its segments
            const Segments sg = segments_of(row, start, p.nt, run);
            float2 x = make_float2(kLowest, 0.f);
            const int hh = threadIdx.x % kHeads;
            if (hh < heads)
                for (long long i = threadIdx.x / kHeads; i < sg.count; i += kCompute / kHeads) {
                    const float2 y = __ldcg(&g.s.stats[(sg.first + i) * g.sp.zg + hh]);
                    if (raw) x = join_pair(x, y);
                    else x = make_float2(isnan(x.x) || isnan(y.x) ? NAN : fmaxf(x.x, y.x), x.y + y.y);
                }
#pragma unroll
            for (int o = 8; o < 32; o <<= 1) {
                const float2 y = make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o));
                if (raw) x = join_pair(x, y);
                else x = make_float2(isnan(x.x) || isnan(y.x) ? NAN : fmaxf(x.x, y.x), x.y + y.y);
            }
            compute_sync();
            if (lane < kHeads) sh.red[warp][lane] = x;
            compute_sync();
            if (threadIdx.x < kHeads) {
                x = sh.red[0][threadIdx.x];
                for (int w = 1; w < kWarps; ++w) {
                    const float2 y = sh.red[w][threadIdx.x];
                    if (raw) x = join_pair(x, y);
                    else x = make_float2(isnan(x.x) || isnan(y.x) ? NAN : fmaxf(x.x, y.x), x.y + y.y);
                }
                const float4 r = row_constants(mode, p.n, x.x, x.y);
                sh.rowc[threadIdx.x] = r;
                if (p.tile == 0 && threadIdx.x < heads) g.s.rowc[row * g.sp.zg + threadIdx.x] = r;
            }
            compute_sync();
            rc = sh.rowc[head];
        }
        float o[PHASE == kScores ? 1 : D / 8][4];
        if constexpr (PHASE != kScores) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        }
        float m = kLowest, sum = 0.f;   // running maximum (softmax: the exponent's reference) and sum of phi or w
        bool bad = false;
        float *zrow = g.s.z + (p.t * g.sp.zg + head) * kTile + 16 * warp + 2 * c4;
        const long long zstep = (long long)g.sp.zg * kTile;
        float2 znext[2];
        if (PHASE == kValues && mine) {
            znext[0] = __ldcg(reinterpret_cast<const float2 *>(zrow));
            znext[1] = __ldcg(reinterpret_cast<const float2 *>(zrow + 8));
        }
        for (int i = 0; i < cnt; ++i) {
            const int left = p.n - (p.tile + i) * kTile;   // keys of the row from this tile on
            float2 z[2], w[2];
            if (PHASE != kValues) {
                const int s = it % C::kStages;
                const bool ok = __all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh.full[s]), (it / C::kStages) & 1, &sh, c.err, kErrFull, true));
                ++it;
                bad |= !ok || sh.bad[s];
                score_tile<T, D>(ring + s * C::kStageBytes, qf, scale, raw, z);
                __syncwarp();
                if (lane == 0 && ok) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[s]));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int j = 16 * warp + 8 * u + 2 * c4;
                    if (j >= left) z[u].x = -INFINITY;
                    if (j + 1 >= left) z[u].y = -INFINITY;
                }
                if (mine && (PHASE == kScores || g.a.scores)) {
                    *reinterpret_cast<float2 *>(zrow) = z[0];
                    *reinterpret_cast<float2 *>(zrow + 8) = z[1];
                }
                zrow += zstep;
            }
            if (PHASE == kScores) {
                const float top = fmaxf(fmaxf(z[0].x, z[0].y), fmaxf(z[1].x, z[1].y)), mn = fmaxf(m, top);
                if (raw) sum *= ptx::ex2(m - mn);
                m = mn;
                sum += (phi(mode, z[0].x, m) + phi(mode, z[0].y, m)) + (phi(mode, z[1].x, m) + phi(mode, z[1].y, m));
                continue;
            }
            if (PHASE == kValues) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    z[u] = znext[u];
                    const int j = 16 * warp + 8 * u + 2 * c4;
                    w[u].x = mine && j < left ? weight(mode, p_exp, z[u].x, rc) : 0.f;
                    w[u].y = mine && j + 1 < left ? weight(mode, p_exp, z[u].y, rc) : 0.f;
                }
                if (i + 1 < cnt && mine) {
                    zrow += zstep;
                    znext[0] = __ldcg(reinterpret_cast<const float2 *>(zrow));
                    znext[1] = __ldcg(reinterpret_cast<const float2 *>(zrow + 8));
                }
            } else if (mode == kSoftmax) {
                // weights 2^(z - m); m follows the maximum only when it has grown by more
                // than 8, so that weights stay below 2^8 and rescaling is rare
                float top = fmaxf(fmaxf(z[0].x, z[0].y), fmaxf(z[1].x, z[1].y));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const bool grow = top > m + 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float mn = grow ? top : m, f = ptx::ex2(m - mn);
                    m = mn;
                    sum *= f;
#pragma unroll
                    for (int k = 0; k < D / 8; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[k][e] *= f;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) w[u] = make_float2(ptx::ex2(z[u].x - m), ptx::ex2(z[u].y - m));
            } else {
#pragma unroll
                for (int u = 0; u < 2; ++u) w[u] = make_float2(phi(mode, z[u].x, 0.f), phi(mode, z[u].y, 0.f));
            }
            sum += (w[0].x + w[0].y) + (w[1].x + w[1].y);
            if constexpr (PHASE != kScores) {
                const int s = it % C::kStages;
                const bool ok = __all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh.full[s]), (it / C::kStages) & 1, &sh, c.err, kErrFull, true));
                ++it;
                bad |= !ok || sh.bad[s];
                value_tile<T, D>(ring + s * C::kStageBytes, w, left, o);
                __syncwarp();
                if (lane == 0 && ok) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[s]));
            }
        }
        // the segment's statistics and sums: the four lanes of a head, then the warps
        const bool relative = PHASE == kScores ? raw : mode == kSoftmax;
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            const float2 y = make_float2(__shfl_xor_sync(0xffffffffu, m, x), __shfl_xor_sync(0xffffffffu, sum, x));
            if (PHASE == kScores && relative) {
                const float2 r = join_pair(make_float2(m, sum), y);
                m = r.x;
                sum = r.y;
            } else {   // the lanes of a head share m in the other phases
                m = fmaxf(m, y.x);
                sum += y.y;
            }
        }
        if (PHASE != kScores && !relative) m = 0.f;
        compute_sync();
        if (c4 == 0) sh.red[warp][head] = make_float2(bad ? NAN : m, sum);
        compute_sync();
        float2 all = sh.red[0][head];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float2 y = sh.red[w][head];
            if (relative) all = join_pair(all, y);
            else all = make_float2(isnan(all.x) || isnan(y.x) ? NAN : fmaxf(all.x, y.x), all.y + y.y);
        }
        if (warp == 0 && c4 == 0 && mine) (PHASE == kScores ? g.s.stats : g.s.sums)[seg * g.sp.zg + head] = all;
        if constexpr (PHASE != kScores) {
            const float f = relative ? ptx::ex2(m - all.x) : 1.f;
#pragma unroll
            for (int k = 0; k < D / 8; ++k)
                *reinterpret_cast<float2 *>(&merge[(warp * kHeads + head) * D + 8 * k + 2 * c4]) =
                    make_float2((o[k][0] + o[k][2]) * f, (o[k][1] + o[k][3]) * f);
            compute_sync();
            for (int i = threadIdx.x; i < heads * D / 4; i += kCompute) {
                float4 x = reinterpret_cast<const float4 *>(merge)[i];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 y = reinterpret_cast<const float4 *>(merge)[w * kHeads * D / 4 + i];
                    x.x += y.x;
                    x.y += y.y;
                    x.z += y.z;
                    x.w += y.w;
                }
                reinterpret_cast<float4 *>(g.s.o + seg * g.sp.zg * D)[i] = x;
            }
        }
        p.t += cnt;
        if (p.t < t1) next_row(c, g.sp.heads_rows, p);
    }
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

__device__ __forceinline__ float2 shuffle_xor(float2 x, int o) {
    return make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o));
}

// (reference, sum of w) over the row's segments i = first, first + step, ...
// of the head whose entries start at `at` (the whole warp calls it).
__device__ float2 join_sums(const float2 *at, int zg, long long first, long long count, long long step) {
    float2 x = make_float2(kLowest, 0.f);
    for (long long i = first; i < count; i += step) x = join_pair(x, __ldcg(at + i * zg));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = join_pair(x, shuffle_xor(x, o));
    return x;
}

// Blocks [0, join_blocks): the output rows, `warps_per` warps for each; the
// others: the scores, by equal runs of tiles of the key heads.  Everything
// that the lengths alone decide is done before the wait for the kernel that
// this one depends on; after it come two rounds of loads for an output row (the
// segments' sums, then their value sums) and two for the scores (the row
// constants, then z and the scores, 16 bytes a thread).
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join(const __grid_constant__ Args g, int join_blocks, int warps_per) {
    const PagedCache &c = g.a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = g.a.H / c.Hkv, mode = g.a.mode;
    const long long per_row = tiles_before(c, c.B), total = per_row * g.sp.heads_rows;
    const int run = run_length(g.sp, total);
    if ((int)blockIdx.x < join_blocks) {
        constexpr int kPerLane = D / 32;
        using Vec = typename std::conditional<kPerLane == 4, float4, float2>::type;
        __shared__ Vec part[kJoinWarps][32];
        __shared__ float2 ms[kJoinWarps];
        const int per_block = kJoinWarps / warps_per, sub = warp % warps_per;
        const long long r = (long long)blockIdx.x * per_block + warp / warps_per;
        const bool live = r < (long long)c.B * g.a.H;
        const int b = live ? (int)(r / g.a.H) : 0, hq = (int)(r % g.a.H), h = hq / G, gq = hq % G;
        const int n = live ? paged_len(c, b) : 0, nt = (n + kTile - 1) / kTile;
        const bool usable = live && c.lens[b] == n;
        const long long before = tiles_before(c, b);
        const int hr = h * g.sp.blocks + gq / kHeads;
        Segments sg = {0, 0};
        if (n > 0) sg = segments_of((long long)b * g.sp.heads_rows + hr, before * g.sp.heads_rows + (long long)hr * nt, nt, run);
        const float2 *sums = g.s.sums + sg.first * g.sp.zg + gq % kHeads;
        const float *o = g.s.o + (sg.first * g.sp.zg + gq % kHeads) * D + lane * kPerLane;
        ptx::grid_dependency_wait();
        float acc[kPerLane];
#pragma unroll
        for (int e = 0; e < kPerLane; ++e) acc[e] = 0.f;
        // this warp's segments sub, sub + warps_per, ...
        const float2 x = join_sums(sums, g.sp.zg, sub + (long long)lane * warps_per, sg.count, 32LL * warps_per);
        float m = x.x, sum = x.y;
        for (long long i0 = sub; i0 < sg.count; i0 += 32LL * warps_per) {
            const long long mine = i0 + (long long)lane * warps_per;
            const float f = mine < sg.count ? ptx::ex2(__ldcg(sums + mine * g.sp.zg).x - m) : 0.f;
            const int cnt = (int)min(32LL, (sg.count - i0 + warps_per - 1) / warps_per);
#pragma unroll 8
            for (int i = 0; i < cnt; ++i) {
                const Vec v = __ldcg(reinterpret_cast<const Vec *>(o + (i0 + (long long)i * warps_per) * g.sp.zg * D));
                const float fi = __shfl_sync(0xffffffffu, f, i);
                acc[0] = fmaf(v.x, fi, acc[0]);
                acc[1] = fmaf(v.y, fi, acc[1]);
                if constexpr (kPerLane == 4) {
                    acc[2] = fmaf(v.z, fi, acc[2]);
                    acc[3] = fmaf(v.w, fi, acc[3]);
                }
            }
        }
        if (warps_per > 1) {
            if constexpr (kPerLane == 4) part[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            else part[warp][lane] = make_float2(acc[0], acc[1]);
            if (lane == 0) ms[warp] = make_float2(m, sum);
            __syncthreads();
            if (sub) return;
            float2 all = ms[warp];
            for (int w = 1; w < warps_per; ++w) all = join_pair(all, ms[warp + w]);
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) acc[e] = 0.f;
            for (int w = 0; w < warps_per; ++w) {
                const float f = ptx::ex2(ms[warp + w].x - all.x);
                const Vec v = part[warp + w][lane];
                acc[0] = fmaf(v.x, f, acc[0]);
                acc[1] = fmaf(v.y, f, acc[1]);
                if constexpr (kPerLane == 4) {
                    acc[2] = fmaf(v.z, f, acc[2]);
                    acc[3] = fmaf(v.w, f, acc[3]);
                }
            }
            m = all.x;
            sum = all.y;
        }
        if (!live) return;
        // a length outside the cache: NaN; an empty sequence: zeros
        const float inv = !usable || isnan(m) ? NAN : n == 0 ? 0.f : 1.f / sum;
        uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(g.a.out) + r * D + lane * kPerLane);
#pragma unroll
        for (int e = 0; e < kPerLane; e += 2) out[e / 2] = Elem<T>::pack(acc[e] * inv, acc[e + 1] * inv);
        return;
    }
    // scores: tiles numbered through (sequence, key head, tile)
    __shared__ float4 rowc[kMaxGroup];
    const long long keys_total = per_row * c.Hkv, cta = (long long)blockIdx.x - join_blocks, ctas = (long long)gridDim.x - join_blocks;
    const long long srun = (keys_total + ctas - 1) / ctas;
    const long long t0 = cta * srun, t1 = t0 + srun < keys_total ? t0 + srun : keys_total;
    Place p = {};
    if (t0 < t1) p = locate(c, c.Hkv, t0);
    p.t = t0;
    const bool vec = ((reinterpret_cast<uintptr_t>(g.a.scores) | reinterpret_cast<uintptr_t>(g.a.scores_out)) & 15) == 0;
    ptx::grid_dependency_wait();
    while (p.t < t1) {
        const int cnt = (int)(t1 - p.t < p.nt - p.tile ? t1 - p.t : p.nt - p.tile);
        // number of the row's first tile among the stream's: the rows before it, each `blocks` times
        const long long start = (p.t - p.tile - (long long)p.hr * p.nt) * g.sp.blocks + (long long)p.hr * g.sp.blocks * p.nt;
        __syncthreads();
        // constants of the G query heads: a warp for each in turn
        for (int gq = warp; gq < G; gq += kJoinWarps) {
            const long long row = (long long)p.b * g.sp.heads_rows + p.hr * g.sp.blocks + gq / kHeads;
            const Segments sg = segments_of(row, start + (long long)(gq / kHeads) * p.nt, p.nt, run);
            float4 r = make_float4(0.f, 1.f, 0.f, 0.f);
            if (is_reweight(mode)) r = __ldcg(&g.s.rowc[row * g.sp.zg + gq % kHeads]);
            const float2 x = join_sums(g.s.sums + sg.first * g.sp.zg + gq % kHeads, g.sp.zg, lane, sg.count, 32);
            if (!is_reweight(mode)) r.x = x.x;
            r.w = isnan(x.x) ? NAN : 1.f / x.y;
            if (lane == 0) rowc[gq] = r;
        }
        __syncthreads();
        // 16 threads per tile, four slots each
        constexpr int kGroups = kJoinThreads / 16;
        const int slot0 = (threadIdx.x % 16) * 4;
        const size_t base = ((size_t)p.b * c.Hkv + p.hr) * c.capacity();
        for (int i = threadIdx.x / 16; i < cnt; i += kGroups) {
            const int slot = (p.tile + i) * kTile + slot0, have = p.n - slot;
            if (have <= 0) continue;
            const float *from = g.a.scores + base + slot;
            float *to = g.a.scores_out + base + slot;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (vec && have >= 4) {
                s = __ldcg(reinterpret_cast<const float4 *>(from));
            } else {
                s.x = from[0];
                if (have > 1) s.y = from[1];
                if (have > 2) s.z = from[2];
                if (have > 3) s.w = from[3];
            }
            float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int gq = 0; gq < G; ++gq) {
                const long long tile = start + (long long)(gq / kHeads) * p.nt + p.tile + i;
                const float4 z = __ldcg(reinterpret_cast<const float4 *>(&g.s.z[(tile * g.sp.zg + gq % kHeads) * kTile + slot0]));
                const float4 rc = rowc[gq];
                add.x = fmaf(weight(mode, g.a.p, z.x, rc), rc.w, add.x);
                add.y = fmaf(weight(mode, g.a.p, z.y, rc), rc.w, add.y);
                add.z = fmaf(weight(mode, g.a.p, z.z, rc), rc.w, add.z);
                add.w = fmaf(weight(mode, g.a.p, z.w, rc), rc.w, add.w);
            }
            s.x += add.x;
            s.y += add.y;
            s.z += add.z;
            s.w += add.w;
            if (vec && have >= 4) {
                *reinterpret_cast<float4 *>(to) = s;
            } else {
                to[0] = s.x;
                if (have > 1) to[1] = s.y;
                if (have > 2) to[2] = s.z;
                if (have > 3) to[3] = s.w;
            }
        }
        p.t += cnt;
        if (p.t < t1) next_row(c, c.Hkv, p);
    }
}

struct Layout {
    Split sp;
    size_t z, stats, sums, o, rowc, total;
};

Layout layout(const PagedDecode &pr, int sms) {
    const PagedCache &c = pr.c;
    const int G = pr.H / c.Hkv;
    Layout l;
    l.sp.blocks = (G + kHeads - 1) / kHeads;
    l.sp.heads_rows = c.Hkv * l.sp.blocks;
    l.sp.zg = G < kHeads ? G : kHeads;
    l.sp.min_run = 1;
    const long long rows = (long long)c.B * l.sp.heads_rows, row_tiles = (c.capacity() + kTile - 1) / kTile;
    const long long most = rows * row_tiles, wave = (long long)sms * (c.d == 64 ? 4 : 3);
    l.sp.ctas = (int)(most < wave ? most : wave);
    const size_t segments = (size_t)rows + l.sp.ctas;
    auto r = [](size_t x) { return (x + 255) & ~(size_t)255; };
    l.z = 0;
    l.stats = is_reweight(pr.mode) || pr.scores ? r((size_t)most * l.sp.zg * kTile * 4) : 0;
    l.sums = l.stats + r(segments * l.sp.zg * 8);
    l.o = l.sums + r(segments * l.sp.zg * 8);
    l.rowc = l.o + r(segments * l.sp.zg * c.d * 4);
    l.total = l.rowc + r((size_t)rows * l.sp.zg * 16);
    return l;
}

cudaError_t launch_dependent(const void *fn, dim3 grid, int block, size_t smem, bool dependent, void **args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

template <typename T, int D, int PHASE>
cudaError_t stream_phase(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int piece_rows, bool dependent, cudaStream_t stream) {
    using C = Config<D, PHASE>;
    constexpr int smem = 1024 + C::kStages * C::kStageBytes + C::kMerge;
    static PerDeviceOnce once;
    const void *fn = (const void *)paged_stream<T, D, PHASE>;
    const cudaError_t e = per_device_once(once, nullptr, [&](int &) { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    void *args[] = {(void *)&km, (void *)&vm, (void *)&g, (void *)&piece_rows};
    return launch_dependent(fn, dim3(g.sp.ctas), kBlock, smem, dependent, args, stream);
}

template <typename T, int D>
cudaError_t launch(const Args &g, const CUtensorMap &km, const CUtensorMap &vm, int piece_rows, cudaStream_t stream) {
    cudaError_t e;
    if (is_reweight(g.a.mode)) {
        e = stream_phase<T, D, kScores>(km, vm, g, piece_rows, false, stream);
        if (e == cudaSuccess) e = stream_phase<T, D, kValues>(km, vm, g, piece_rows, true, stream);
    } else {
        e = stream_phase<T, D, kBoth>(km, vm, g, piece_rows, false, stream);
    }
    if (e != cudaSuccess) return e;
    // output rows: a whole block for each while a row has many segments
    const long long rows = (long long)g.a.c.B * g.a.H;
    int warps_per = g.sp.ctas >= 16LL * g.a.c.B * g.sp.heads_rows ? kJoinWarps : 1;
    int join_blocks = (int)((rows * warps_per + kJoinWarps - 1) / kJoinWarps);
    const int blocks = join_blocks + (g.a.scores ? g.sp.ctas : 0);
    void *args[] = {(void *)&g, (void *)&join_blocks, (void *)&warps_per};
    return launch_dependent((const void *)paged_join<T, D>, dim3(blocks), kJoinThreads, 0, true, args, stream);
}

}  // namespace

size_t paged_decode_workspace_bytes(const PagedDecode &pr, int sms) { return layout(pr, sms).total; }

cudaError_t launch_paged_decode(const PagedDecode &pr, void *ws, int sms, cudaStream_t stream) {
    Args g;
    g.a = pr;
    cudaError_t e = error_word_ptr(&g.a.c.err);
    if (e != cudaSuccess) return e;
    const PagedCache &c = pr.c;
    const Layout l = layout(pr, sms);
    g.sp = l.sp;
    char *base = static_cast<char *>(ws);
    g.s.z = reinterpret_cast<float *>(base + l.z);
    g.s.stats = reinterpret_cast<float2 *>(base + l.stats);
    g.s.sums = reinterpret_cast<float2 *>(base + l.sums);
    g.s.o = reinterpret_cast<float *>(base + l.o);
    g.s.rowc = reinterpret_cast<float4 *>(base + l.rowc);
    // a copy takes the rows of one page that lie in one tile: the largest power
    // of two that divides the page size, so that no copy crosses either border
    const int low = c.page_size & -c.page_size, piece_rows = low < kTile ? low : kTile;
    CUtensorMap km, vm;
    if (!make_page_map(&km, c.k, c.half, c.d, c.Hkv * c.page_size, c.n_pages, c.page_stride, piece_rows) ||
        !make_page_map(&vm, c.v, c.half, c.d, c.Hkv * c.page_size, c.n_pages, c.page_stride, piece_rows))
        return cudaErrorInvalidValue;
    if (c.half) return c.d == 64 ? launch<__half, 64>(g, km, vm, piece_rows, stream) : launch<__half, 128>(g, km, vm, piece_rows, stream);
    return c.d == 64 ? launch<__nv_bfloat16, 64>(g, km, vm, piece_rows, stream) : launch<__nv_bfloat16, 128>(g, km, vm, piece_rows, stream);
}

}  // namespace lssar
