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
// Split.  The tokens of all sequences are cut into tiles of 16 KB of one key
// head, numbered through (sequence, key head, block of 8 query heads, tile), and
// the tiles into chunks wherever rows begin or end, so that lengths of any mix
// load the SMs evenly; the part of a row inside one chunk is a segment.  The
// lengths are on the device: each warp finds its places by a prefix sum.  CTAs
// take chunks by tickets:
//   softmax, LSSA: K and V tiles in one pass, softmax weights relative to a
//                  running maximum.  Without scores, one large chunk per CTA and
//                  then small ones: the SMs do not get equal shares of the
//                  memory's bandwidth (equal chunks ended between 56 and 104 us
//                  on one ragged batch);
//   re-weighting:  K tiles -> z (scratch) and (m, S1) of each segment; when no
//                  chunk is left, each CTA takes its own again: the row
//                  constants, once all segments of the row are in, z -> w, V tiles;
//   then           scores: each CTA its own chunks once more, row by row as the
//                  rows' sums are in.
// A row that lies in one chunk is written at once; one of a few segments by the
// CTA that finishes it; one of many by a CTA per query head.  What a CTA waits for
// has been taken before by a running CTA that does not wait for this one: no
// launch order or residency is needed for progress.  A producer warp takes the
// tickets and streams the tiles ahead of the compute warps.
//
// Products on mma.sync m16n8k16: a decode row has G <= 8 query heads per key head
// in a block, which a 128-row tcgen05 tile would leave almost empty, and the
// tensor work is a small part of the time that HBM needs.  The 16 rows of an
// operand carry the 8 heads and, for free, something else that is needed:
//   scores: rows 8-15 the queries, rows 0-7 the tile's own 8 keys, so that one
//           product gives q.k and, on the diagonal, |k|^2;
//   values: rows 8-15 the weights rounded to 16 bits, rows 0-7 what the rounding
//           left over, so that weights keep 16 bits (bf16) or more.
// K and V tiles come by TMA (128-byte swizzle), a piece of a page at a time.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "paged.cuh"
#include "row_weights.cuh"
#include "tc_host.cuh"
#include "tc_ptx.cuh"

namespace lssar {
namespace paged {

constexpr int kWarps = 4;                     // compute warps, each a quarter of every tile's keys
constexpr int kCompute = kWarps * 32;
constexpr int kBlock = kCompute + 32;         // + the producer warp
constexpr int kHeads = 8;                     // query heads per block of heads
constexpr int kMaxGroup = 128;                // H / Hkv
constexpr int kMaxCtas = 1024;
constexpr int kFewSegments = 16;              // rows of at most so many are joined by the CTA that finishes them
constexpr float kLowest = -3.0e38f;           // below every score, and finite
constexpr uint64_t kWaitLimitNs = 2000000000ull;
enum : unsigned { kErrFull = 53, kErrEmpty, kErrDrain, kErrCount, kErrItem };

constexpr int tile_keys(int d) { return 8192 / d; }   // 16 KB of K or V

// Shared memory: the ring of tiles, and per warp the sums of w v at a
// segment's end (before it, the weights of a batch of tiles).  Three or four
// CTAs per SM: segments' ends and beginnings overlap.
template <int D>
struct Config {
    static constexpr int kTile = tile_keys(D);
    static constexpr int kKeys = kTile / kWarps;       // keys per warp and tile
    static constexpr int kEights = kKeys / 8;          // blocks of 8 keys
    static constexpr int kPairs = kKeys / 2;           // pairs of keys per warp and tile
    static constexpr int kBatch = 32 / kPairs;         // tiles whose weights are formed together (32 pairs)
    static constexpr int kStageBytes = kTile * D * 2;
    static constexpr int kStages = 3;
    static constexpr int kPerSm = D == 64 ? 3 : 3;
    static constexpr int kMerge = kWarps * kHeads * D * 4;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kMerge;
};
constexpr int kMaxStages = 8;

// How a launch is laid out.
struct Split {
    int heads_rows;        // Hkv * blocks: rows per sequence
    int blocks;            // blocks of kHeads query heads per key head
    int zg;                // heads stored per tile: min(G, kHeads)
    int ctas;              // CTAs
    int rows;              // B * heads_rows
};

struct Scratch {
    float *z;              // [tile][zg][keys]: z, then w (re-weighting with scores)
    float2 *stats;         // [segment][zg]: max of z, sum of phi
    float2 *sums;          // [segment][zg]: reference of the exponent (softmax), sum of w
    float *o;              // [segment][zg][D]: sum of w v
    unsigned *next;        // tickets handed out; zero at launch, as are:
    unsigned *scored;      // [row] segments with z and stats written
    unsigned *summed;      // [row] segments with sums and o written
};

struct Args {
    PagedDecode a;
    Split sp;
    Scratch s;
    int piece_rows;        // rows of a page per copy
};

// A place in the numbering of the tiles.
struct Place {
    int t;                 // number of the tile
    int b, hr, tile;       // sequence, row of the sequence, tile of the row
    int n, nt;             // length and tiles of the sequence
};

template <int D>
__device__ __forceinline__ int tiles_of(int n) {
    return (n + Config<D>::kTile - 1) / Config<D>::kTile;
}

// Tiles of sequences [0, upto) for one row of each, and those of the longest
// (the whole warp calls it).
template <int D>
__device__ int tiles_before(const PagedCache &c, int upto, int *longest = nullptr) {
    int x = 0, most = 0;
    for (int b = threadIdx.x & 31; b < upto; b += 32) {
        const int nt = tiles_of<D>(paged_len(c, b));
        x += nt;
        most = max(most, nt);
    }
    if (longest) *longest = __reduce_max_sync(0xffffffffu, most);
    return __reduce_add_sync(0xffffffffu, x);
}

// The chunks of `total` tiles: equal ones, one per CTA, or one of `big` tiles for
// each CTA, 3/4 of an equal share, and then about two `small` ones per CTA, whose
// order of finishing evens out the SMs' rates.  (With few tiles per CTA the end of
// a segment costs as much as some tiles: equal chunks.)
struct Chunks {
    int total, big, ctas, small;
    __device__ __forceinline__ Chunks(int tiles, int n, bool equal) : total(tiles), ctas(n) {
        const int share = tiles / n;
        big = equal || share < 6 ? 0 : share * 3 / 4;
        const int rest = tiles - big * n, parts = big ? 2 * n : n;
        small = max(1, (rest + parts - 1) / parts);
    }
    __device__ __forceinline__ int of(int t) const { return t < big * ctas ? t / big : (big ? ctas : 0) + (t - big * ctas) / small; }
    __device__ __forceinline__ int count() const { return total ? of(total - 1) + 1 : 0; }
    __device__ __forceinline__ int begin(int i) const { return big && i < ctas ? i * big : big * ctas + (i - (big ? ctas : 0)) * small; }
    __device__ __forceinline__ int end(int i) const { return min(total, begin(i) + (big && i < ctas ? big : small)); }
};
constexpr int kChunksPerCta = 3;   // at most, and one more

// The place of tile t < total (the whole warp calls it).
template <int D>
__device__ Place locate(const PagedCache &c, int rows_per_seq, int t) {
    const int lane = threadIdx.x & 31;
    Place p;
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < c.B ? paged_len(c, b) : 0, nt = tiles_of<D>(n);
        int end = nt * rows_per_seq;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + end > t);
        if (hit) {
            const int l = __ffs(hit) - 1;
            p.n = __shfl_sync(0xffffffffu, n, l);
            p.nt = __shfl_sync(0xffffffffu, nt, l);
            const int in = t - (before + __shfl_sync(0xffffffffu, end, l) - p.nt * rows_per_seq);
            p.b = b0 + l;
            p.hr = in / p.nt;
            p.tile = in % p.nt;
            p.t = t;
            return p;
        }
        before += __shfl_sync(0xffffffffu, end, 31);
    }
}

// On to the first tile of the next row that has one.
template <int D>
__device__ __forceinline__ void next_row(const PagedCache &c, int rows_per_seq, Place &p) {
    p.tile = 0;
    if (++p.hr < rows_per_seq) return;
    p.hr = 0;
    do {
        if (++p.b >= c.B) return;
        p.n = paged_len(c, p.b);
        p.nt = tiles_of<D>(p.n);
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
template <int D>
__device__ __forceinline__ uint32_t piece(uint32_t tile, int row, int chunk) {
    return tile + (chunk >> 3) * (Config<D>::kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory"); }

// A work item as the producer hands it to the compute warps.
enum Kind : int { kScoreTiles, kValueTiles, kAddScores, kJoinRow, kEnd };
struct Item {
    Place p;
    int t1, kind, index;
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t item_full[2], item_empty[2];
    Item item[2];
    unsigned short mine[kMaxCtas];  // the chunks of this CTA
    int bad[kMaxStages];            // the stage's tile names a page that is none
    float2 red[kWarps][kHeads];
    float4 rowc[kMaxGroup];         // row constants: m, kappa, beta; for the scores: m, 1 / sum of w
    int last;                       // this CTA has finished a row
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

// The segments of the row that starts at tile `start`: `count` from chunk
// `chunk` on, with scratch entries first, first + 1, ... = row + chunk (both grow
// along the numbering, so that no two segments share one).
struct Segments {
    int first, count;
};
__device__ __forceinline__ Segments segments_of(const Chunks &ch, int row, int start, int nt) {
    const int a = ch.of(start), b = ch.of(start + nt - 1);
    return Segments{row + a, b - a + 1};
}

// One more segment of a row is in: what this thread has seen written is visible
// to whoever sees the count.
__device__ __forceinline__ void signal(unsigned *count) { asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory"); }

// Waits (bounded) until a row's count is reached; one thread calls it, and what
// was written before the count is visible to the threads that meet it at a barrier.
__device__ inline void wait_count(const unsigned *count, unsigned want, Shared *sh, unsigned *err) {
    // plain polls and one fence: each acquiring load would empty the SM's L1
    if (*(volatile const unsigned *)count < want) {
        const uint64_t t0 = ptx::globaltimer_ns();
        do {
            __nanosleep(100);
            if (*(volatile int *)&sh->abort_flag) break;
            if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
                atomicCAS(err, 0u, (unsigned)kErrCount);
                *(volatile int *)&sh->abort_flag = 1;
                break;
            }
        } while (*(volatile const unsigned *)count < want);
    }
    __threadfence();
}

// (m, s): sums s relative to 2^m.  NaN (a row that must not be used) stays:
// fmaxf alone would drop it.
__device__ __forceinline__ float2 join_pair(float2 x, float2 y) {
    const float m = isnan(x.x) || isnan(y.x) ? NAN : fmaxf(x.x, y.x);
    return make_float2(m, x.y * ptx::ex2(x.x - m) + y.y * ptx::ex2(y.x - m));
}
// (m, s): a maximum and a plain sum.
__device__ __forceinline__ float2 join_plain(float2 x, float2 y) {
    return make_float2(isnan(x.x) || isnan(y.x) ? NAN : fmaxf(x.x, y.x), x.y + y.y);
}
__device__ __forceinline__ float2 shuffle_xor(float2 x, int o) {
    return make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o));
}

// Row constants m, kappa, beta from the row's maximum and normaliser sum.
template <int MODE>
__device__ __forceinline__ float4 row_constants(int n, float m, float s1) {
    const float theta = n <= 3 ? 0.f : s1 / (float)n, top = phi(MODE, m, m), den = top - theta;
    float kappa = 0.f, beta = 1.f;     // all-zero re-weighted row: uniform
    if (den > 1e-5f * top + 2e-5f) {   // the prefill kernel's near-uniform band
        kappa = 1.f / den;
        beta = -theta * kappa;
    }
    if (isnan(m) || isnan(s1)) kappa = NAN;
    return make_float4(m, kappa, beta, 0.f);
}

// x[i]^p for N values at once (independent chains).
template <int N>
__device__ __forceinline__ void powers(float (&x)[N], int p) {
    float r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = p & 1 ? x[i] : 1.f;
    for (p >>= 1; p; p >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= x[i];
        if (p & 1)
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] *= x[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = r[i];
}

// Producer warp: the tiles of an item through the ring, from place p to tile t1.  WHAT: 0 K tiles, 1 V tiles, 2 the K then the V tile of each.
// `it` counts the stages used so far.
template <int D, int WHAT>
__device__ bool produce(const Args &g, const CUtensorMap *km, const CUtensorMap *vm, Shared *sh, uint32_t ring, Place p, int t1, int &it) {
    using C = Config<D>;
    const PagedCache &c = g.a.c;
    const int lane = threadIdx.x & 31, piece_rows = g.piece_rows, pieces = C::kTile / piece_rows;
    // the page of this lane's piece of a tile; -1: past the row's end, -2: none of the pool
    auto look_up = [&](const Place &q) {
        const int s0 = q.tile * C::kTile + lane * piece_rows;
        if (lane >= pieces || s0 >= q.n) return -1;
        const int pg = paged_page(c, q.b, s0 / c.page_size);
        return pg < 0 ? -2 : pg;
    };
    int pg = look_up(p);
    while (true) {
        Place q = p;
        ++q.t;
        int next = -1;
        if (q.t < t1) {
            if (++q.tile == q.nt) next_row<D>(c, g.sp.heads_rows, q);
            next = look_up(q);
        }
        const unsigned ok = __ballot_sync(0xffffffffu, pg >= 0), bad = __ballot_sync(0xffffffffu, pg == -2);
        const int s0 = p.tile * C::kTile + lane * piece_rows;
        const int y = p.hr / g.sp.blocks * c.page_size + s0 % c.page_size;
#pragma unroll
        for (int u = 0; u < (WHAT == 2 ? 2 : 1); ++u, ++it) {
            const int s = it % C::kStages, use = it / C::kStages;
            if (use > 0 && !__all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh->empty[s]), (use - 1) & 1, sh, c.err, kErrEmpty, true)))
                return false;
            const uint32_t full = ptx::smem_u32(&sh->full[s]), dst = ring + s * C::kStageBytes + lane * piece_rows * 128;
            const CUtensorMap *map = WHAT == 1 || u == 1 ? vm : km;
            if (lane == 0) {
                sh->bad[s] = bad != 0;
                ptx::mbar_arrive_expect_tx(full, (uint32_t)__popc(ok) * piece_rows * D * 2);
            }
            __syncwarp();
            if (pg >= 0 && dcheck(y >= 0 && y + piece_rows <= c.Hkv * c.page_size && pg < c.n_pages && lane < pieces, c.err, kDbgTma)) {
                ptx::tma_load_3d(dst, map, full, 0, y, pg);
                if (D == 128) ptx::tma_load_3d(dst + C::kTile * 128, map, full, 64, y, pg);
            }
        }
        if (q.t >= t1) return true;
        p = q;
        pg = next;
    }
}

// The scores z of the warp's keys of a tile (blocks of 8 keys): head lane / 4,
// keys 2 (lane % 4) + {0, 1} of each block.
template <typename T, int D, bool RAW>
__device__ __forceinline__ void score_tile(uint32_t tile, const uint32_t (&qf)[D / 16][2], float scale, float2 (&z)[Config<D>::kEights]) {
    using C = Config<D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int u = 0; u < C::kEights; ++u) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const int row = C::kKeys * warp + 8 * u + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t r[4];
            ldsm4(r, piece<D>(tile, row, 4 * kk + (lane >> 3)));
            Elem<T>::mma(d, r[0], qf[2 * kk][0], r[1], qf[2 * kk][1], r[0], r[1]);
            Elem<T>::mma(d, r[2], qf[2 * kk + 1][0], r[3], qf[2 * kk + 1][1], r[2], r[3]);
        }
        z[u] = make_float2(scale * d[2], scale * d[3]);
        if (!RAW) {
            // |k|^2 of keys 2c and 2c + 1 is on the diagonal: rows 2c, 2c + 1 of the upper half
            const int c = lane & 3;
            const float ka = __shfl_sync(0xffffffffu, d[0], 9 * c), kb = __shfl_sync(0xffffffffu, d[1], 9 * c + 4);
            z[u].x *= rsqrtf(fmaxf(ka, 1e-24f));   // |k| clamped at 1e-12 as everywhere
            z[u].y *= rsqrtf(fmaxf(kb, 1e-24f));
        }
    }
}

// Two weights as operand words: rounded, and what the rounding left over.
template <typename T>
__device__ __forceinline__ uint2 split_weights(float2 w) {
    uint2 r;
    r.x = Elem<T>::pack(w.x, w.y);
    const float2 f = Elem<T>::unpack(r.x);
    r.y = Elem<T>::pack(w.x - f.x, w.y - f.y);
    return r;
}

// Adds w v of the warp's keys of a tile to o (n8 blocks of columns; [0..1] from
// the weights' remainders, [2..3] from the rounded weights).  w[u]: the split
// weights of head lane / 4, keys 2 (lane % 4) + {0, 1} of block u.
template <typename T, int D>
__device__ __forceinline__ void value_tile(uint32_t tile, const uint2 (&w)[Config<D>::kEights], int left, float (&o)[D / 8][4]) {
    using C = Config<D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3;
    // rows at or past `left` of the tile hold anything (0 * NaN): clear them
    const bool tail = left < C::kTile;
#pragma unroll
    for (int ks = 0; ks < C::kEights / 2; ++ks) {
        const int row = C::kKeys * warp + 16 * ks + (lane & 15);
        uint32_t mask[2] = {0xffffffffu, 0xffffffffu};
        if (tail)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = C::kKeys * warp + 16 * ks + 8 * u + 2 * c;
                mask[u] = (j < left ? 0xffffu : 0u) | (j + 1 < left ? 0xffff0000u : 0u);
            }
#pragma unroll
        for (int np = 0; np < D / 16; ++np) {
            uint32_t r[4];
            ldsm4t(r, piece<D>(tile, row, 2 * np + (lane >> 4)));
            if (tail) {
                r[0] &= mask[0];
                r[1] &= mask[1];
                r[2] &= mask[0];
                r[3] &= mask[1];
            }
            Elem<T>::mma(o[2 * np], w[2 * ks].y, w[2 * ks].x, w[2 * ks + 1].y, w[2 * ks + 1].x, r[0], r[1]);
            Elem<T>::mma(o[2 * np + 1], w[2 * ks].y, w[2 * ks].x, w[2 * ks + 1].y, w[2 * ks + 1].x, r[2], r[3]);
        }
    }
}

// The compute warps' side: what every kind of item needs.
template <int D>
struct Worker {
    const Args &g;
    Shared &sh;
    const uint32_t ring;
    float *const merge;
    const Chunks chunks;
    int it = 0;         // stages used so far
    bool bad = false;   // a stage of the segment was unusable

    // waits for the next stage and uses it
    template <class F>
    __device__ __forceinline__ void stage(F &&use) {
        using C = Config<D>;
        const int s = it % C::kStages;
        const bool ok = __all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh.full[s]), (it / C::kStages) & 1, &sh, g.a.c.err, kErrFull, true));
        ++it;
        bad |= !ok || sh.bad[s];
        use(ring + s * C::kStageBytes);
        __syncwarp();
        if ((threadIdx.x & 31) == 0 && ok) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[s]));
    }
};

// One segment of a row.
struct Segment {
    int row, at;            // the row, and the segment's entry in scratch
    Segments all;           // all of the row's
    int cnt, g0, heads;     // tiles, first query head of the block, query heads
};

__device__ __forceinline__ Segment segment_at(const Args &g, const Chunks &ch, const Place &p, int t1) {
    Segment s;
    s.row = p.b * g.sp.heads_rows + p.hr;
    s.all = segments_of(ch, s.row, p.t - p.tile, p.nt);
    s.at = s.row + ch.of(p.t);
    s.cnt = min(t1 - p.t, p.nt - p.tile);
    s.g0 = p.hr % g.sp.blocks * kHeads;
    s.heads = min(kHeads, g.a.H / g.a.c.Hkv - s.g0);
    return s;
}

// Query fragments of a segment (rows past the block's heads are zero) and the
// factor of its scores; asks for the next row's queries.
template <typename T, int D, bool RAW>
__device__ float load_queries(const Args &g, const Place &p, const Segment &s, int t1, uint32_t (&qf)[D / 16][2]) {
    const int lane = threadIdx.x & 31, head = lane >> 2, c4 = lane & 3, G = g.a.H / g.a.c.Hkv;
    auto row = [&](const Place &x) {
        return static_cast<const uint16_t *>(g.a.q) + x.b * g.a.q_b + (x.hr / g.sp.blocks * G + x.hr % g.sp.blocks * kHeads + head) * g.a.q_h;
    };
    const uint16_t *q = row(p);
    float ss = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int u = 0; u < 2; ++u) qf[kk][u] = head < s.heads ? *reinterpret_cast<const uint32_t *>(q + 16 * kk + 8 * u + 2 * c4) : 0u;
    if (p.t + s.cnt < t1) {
        Place x = p;
        next_row<D>(g.a.c, g.sp.heads_rows, x);
        if (x.hr % g.sp.blocks * kHeads + head < G) asm volatile("prefetch.global.L1 [%0];" ::"l"(row(x) + c4 * (D / 4)));
    }
    if (RAW) return 1.4426950408889634f * rsqrtf((float)D);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float2 x = Elem<T>::unpack(qf[kk][u]);
            ss += x.x * x.x + x.y * x.y;
        }
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    return 1.4426950408889634f * logf((float)D) * logf((float)p.n) / fmaxf(sqrtf(ss), 1e-12f);
}

// The next tile's scores, -inf past the row's end (left: keys of the row from
// the tile on), written to zrow where it is not null.
template <typename T, int D, bool RAW>
__device__ __forceinline__ void next_scores(Worker<D> &w, const uint32_t (&qf)[D / 16][2], float scale, int left, float *zrow, float2 (&z)[Config<D>::kEights]) {
    using C = Config<D>;
    w.stage([&](uint32_t tile) { score_tile<T, D, RAW>(tile, qf, scale, z); });
    if (left < C::kTile) {
        const int j = C::kKeys * (threadIdx.x >> 5) + 2 * (threadIdx.x & 3);
#pragma unroll
        for (int u = 0; u < C::kEights; ++u) {
            if (j + 8 * u >= left) z[u].x = -INFINITY;
            if (j + 8 * u + 1 >= left) z[u].y = -INFINITY;
        }
    }
    if (zrow)
#pragma unroll
        for (int u = 0; u < C::kEights; ++u) *reinterpret_cast<float2 *>(zrow + 8 * u) = z[u];
}

// The statistics of a segment over the warps, from each head's in its four
// lanes: on return in every lane of the head, and in dst.
template <bool RELATIVE>
__device__ __forceinline__ float2 warps_join(Shared &sh, float2 x, bool bad, float2 *dst, int heads) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = lane >> 2;
    compute_sync();
    if ((lane & 3) == 0) sh.red[warp][head] = make_float2(bad ? NAN : x.x, x.y);
    compute_sync();
    x = sh.red[0][head];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) x = RELATIVE ? join_pair(x, sh.red[w][head]) : join_plain(x, sh.red[w][head]);
    if (warp == 0 && (lane & 3) == 0 && head < heads) dst[head] = x;
    return x;
}

// The end of a segment's values: sums of w and w v over the warps; a row with
// this segment alone is written out, the others go to scratch.
template <typename T, int D, bool RELATIVE>
__device__ void finish_values(Worker<D> &w, const Place &p, const Segment &s, float m, float sum, const float (&o)[D / 8][4]) {
    const Args &g = w.g;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = lane >> 2, c4 = lane & 3;
    const long long seg = s.at;
    const float2 all = warps_join<RELATIVE>(w.sh, make_float2(m, sum), w.bad, g.s.sums + seg * g.sp.zg, s.heads);
    const bool whole = s.all.count == 1;
    // softmax sums come to the joint reference; a row's only segment is normalised here
    float f = RELATIVE ? ptx::ex2(m - all.x) : 1.f;
    if (whole) f = isnan(all.x) ? NAN : f / all.y;
#pragma unroll
    for (int k = 0; k < D / 8; ++k)
        *reinterpret_cast<float2 *>(&w.merge[(warp * kHeads + head) * D + 8 * k + 2 * c4]) =
            make_float2((o[k][0] + o[k][2]) * f, (o[k][1] + o[k][3]) * f);
    compute_sync();
    const int hq = p.hr / g.sp.blocks * (g.a.H / g.a.c.Hkv) + s.g0;
    uint16_t *out = static_cast<uint16_t *>(g.a.out) + ((long long)p.b * g.a.H + hq) * D;
    for (int i = threadIdx.x; i < s.heads * D / 4; i += kCompute) {
        float4 x = reinterpret_cast<const float4 *>(w.merge)[i];
#pragma unroll
        for (int u = 1; u < kWarps; ++u) {
            const float4 y = reinterpret_cast<const float4 *>(w.merge)[u * kHeads * D / 4 + i];
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
        }
        if (whole) reinterpret_cast<uint2 *>(out)[i] = make_uint2(Elem<T>::pack(x.x, x.y), Elem<T>::pack(x.z, x.w));
        else reinterpret_cast<float4 *>(g.s.o + seg * g.sp.zg * D)[i] = x;
    }
    if (whole) {
        // (the scores of a group of several blocks are added by one of them)
        if (g.a.scores && g.sp.blocks > 1) {
            compute_sync();
            if (threadIdx.x == 0) signal(g.s.summed + s.row);
        }
        return;
    }
    const bool few = s.all.count <= kFewSegments;
    compute_sync();
    if (threadIdx.x == 0) {
        if (few) {
            __threadfence();
            w.sh.last = atomicAdd(g.s.summed + s.row, 1u) == (unsigned)s.all.count - 1;
            __threadfence();
        } else {
            signal(g.s.summed + s.row);
        }
    }
    if (!few) return;
    compute_sync();
    if (!w.sh.last) return;
    // the row's segments in their order, whoever finished last
    const float2 *sums = g.s.sums + (long long)s.all.first * g.sp.zg;
    const float *from = g.s.o + (long long)s.all.first * g.sp.zg * D;
    for (int i = threadIdx.x; i < s.heads * D / 4; i += kCompute) {
        const int hh = i / (D / 4);
        float2 total = make_float2(kLowest, 0.f);
        for (int k = 0; k < s.all.count; ++k) total = RELATIVE ? join_pair(total, __ldcg(sums + k * g.sp.zg + hh)) : join_plain(total, __ldcg(sums + k * g.sp.zg + hh));
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < s.all.count; ++k) {
            const float f = RELATIVE ? ptx::ex2(__ldcg(sums + k * g.sp.zg + hh).x - total.x) : 1.f;
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(from + (long long)k * g.sp.zg * D) + i);
            x.x = fmaf(y.x, f, x.x);
            x.y = fmaf(y.y, f, x.y);
            x.z = fmaf(y.z, f, x.z);
            x.w = fmaf(y.w, f, x.w);
        }
        const float inv = isnan(total.x) ? NAN : 1.f / total.y;
        reinterpret_cast<uint2 *>(out)[i] = make_uint2(Elem<T>::pack(x.x * inv, x.y * inv), Elem<T>::pack(x.z * inv, x.w * inv));
    }
}

// Softmax and LSSA: a segment's scores and values in one pass.
template <typename T, int D, int MODE>
__device__ void one_pass_segment(Worker<D> &w, const Place &p, const Segment &s, int t1) {
    using C = Config<D>;
    constexpr bool kRaw = MODE == kSoftmax;
    const Args &g = w.g;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = lane >> 2, c4 = lane & 3;
    uint32_t qf[D / 16][2];
    const float scale = load_queries<T, D, kRaw>(g, p, s, t1, qf);
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m = MODE == kSoftmax ? kLowest : 0.f, sum = 0.f;
    float *zrow = g.a.scores && head < s.heads ? g.s.z + ((long long)p.t * g.sp.zg + head) * C::kTile + C::kKeys * warp + 2 * c4 : nullptr;
    for (int i = 0; i < s.cnt; ++i) {
        const int left = p.n - (p.tile + i) * C::kTile;
        float2 z[C::kEights];
        next_scores<T, D, kRaw>(w, qf, scale, left, zrow, z);
        if (zrow) zrow += g.sp.zg * C::kTile;
        if (MODE == kSoftmax) {
            // weights 2^(z - m); m follows the maximum only when it has grown by more
            // than 8, so that weights stay below 2^8 and rescaling is rare
            float top = fmaxf(z[0].x, z[0].y);
#pragma unroll
            for (int u = 1; u < C::kEights; ++u) top = fmaxf(top, fmaxf(z[u].x, z[u].y));
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
        }
        uint2 ws[C::kEights];
#pragma unroll
        for (int u = 0; u < C::kEights; ++u) {
            const float2 y = make_float2(phi(MODE, z[u].x, m), phi(MODE, z[u].y, m));
            sum += y.x + y.y;
            ws[u] = split_weights<T>(y);
        }
        w.stage([&](uint32_t tile) { value_tile<T, D>(tile, ws, left, o); });
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);   // the lanes of a head share m
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    finish_values<T, D, MODE == kSoftmax>(w, p, s, m, sum, o);
}

// Re-weighting, first pass over a segment: z, max z and sum phi.
template <typename T, int D, int MODE>
__device__ void scores_segment(Worker<D> &w, const Place &p, const Segment &s, int t1) {
    using C = Config<D>;
    constexpr bool kRaw = MODE == kSoftmaxRw;
    const Args &g = w.g;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = lane >> 2, c4 = lane & 3;
    uint32_t qf[D / 16][2];
    const float scale = load_queries<T, D, kRaw>(g, p, s, t1, qf);
    float2 x = make_float2(kLowest, 0.f);
    float *zrow = head < s.heads ? g.s.z + ((long long)p.t * g.sp.zg + head) * C::kTile + C::kKeys * warp + 2 * c4 : nullptr;
    for (int i = 0; i < s.cnt; ++i) {
        float2 z[C::kEights];
        next_scores<T, D, kRaw>(w, qf, scale, p.n - (p.tile + i) * C::kTile, zrow, z);
        if (zrow) zrow += g.sp.zg * C::kTile;
        float top = x.x;
#pragma unroll
        for (int u = 0; u < C::kEights; ++u) top = fmaxf(top, fmaxf(z[u].x, z[u].y));
        if (kRaw) x.y *= ptx::ex2(x.x - top);
        x.x = top;
#pragma unroll
        for (int u = 0; u < C::kEights; ++u) x.y += phi(MODE, z[u].x, top) + phi(MODE, z[u].y, top);
    }
#pragma unroll
    for (int e = 1; e < 4; e <<= 1) x = kRaw ? join_pair(x, shuffle_xor(x, e)) : join_plain(x, shuffle_xor(x, e));
    warps_join<kRaw>(w.sh, x, w.bad, g.s.stats + (long long)s.at * g.sp.zg, s.heads);
    if (warp == 0 && s.all.count > 1) {   // which wrote the statistics
        __syncwarp();
        if (lane == 0) signal(g.s.scored + s.row);
    }
}

// Re-weighting, second pass over a segment: the row's constants, w and sum w v.
template <typename T, int D, int MODE>
__device__ void values_segment(Worker<D> &w, const Place &p, const Segment &s) {
    using C = Config<D>;
    constexpr bool kRaw = MODE == kSoftmaxRw;
    const Args &g = w.g;
    Shared &sh = w.sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = lane >> 2, c4 = lane & 3;
    // Weights of kBatch tiles at a time, in pairs of keys spread over all lanes
    // whatever the number of heads, and to the operand layout through shared
    // memory (the warp's own part of `merge`; the place of a pair is permuted by
    // the head so that the operand reads hit every bank once).
    uint2 *wbuf = reinterpret_cast<uint2 *>(w.merge + warp * kHeads * D);
    const int bi = lane / C::kPairs, bj = C::kKeys * warp + 2 * (lane % C::kPairs);   // tile of the batch, first key
    float *zl = g.s.z + (long long)(p.t + bi) * g.sp.zg * C::kTile + bj;
    float2 zn[kHeads];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int x = 0; x < kHeads; ++x)
            if (x < s.heads && i0 + bi < s.cnt) zn[x] = __ldcg(reinterpret_cast<const float2 *>(zl + ((long long)i0 * g.sp.zg + x) * C::kTile));
    };
    if (threadIdx.x == 0 && s.all.count > 1) wait_count(g.s.scored + s.row, (unsigned)s.all.count, &sh, g.a.c.err);
    fetch(0);   // the CTA's own
    // the row's constants: 16 threads per head over its segments
    {
        compute_sync();
        float2 x = make_float2(kLowest, 0.f);
        const int hh = threadIdx.x % kHeads;
        const float2 *at = g.s.stats + (long long)s.all.first * g.sp.zg + hh;
        if (hh < s.heads)
#pragma unroll 8
            for (int i = threadIdx.x / kHeads; i < s.all.count; i += kCompute / kHeads) {
                const float2 y = __ldcg(at + (long long)i * g.sp.zg);
                x = kRaw ? join_pair(x, y) : join_plain(x, y);
            }
#pragma unroll
        for (int e = 8; e < 32; e <<= 1) x = kRaw ? join_pair(x, shuffle_xor(x, e)) : join_plain(x, shuffle_xor(x, e));
        compute_sync();
        if (lane < kHeads) sh.red[warp][lane] = x;
        compute_sync();
        if (threadIdx.x < kHeads) {
            x = sh.red[0][threadIdx.x];
            for (int u = 1; u < kWarps; ++u) x = kRaw ? join_pair(x, sh.red[u][threadIdx.x]) : join_plain(x, sh.red[u][threadIdx.x]);
            sh.rowc[threadIdx.x] = row_constants<MODE>(p.n, x.x, x.y);
        }
        compute_sync();
    }
    float o[D / 8][4], wsum[kHeads];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
    for (int x = 0; x < kHeads; ++x) wsum[x] = 0.f;
    for (int i0 = 0; i0 < s.cnt; i0 += C::kBatch) {
        // keys of the row from the lane's first on; none in a tile past the segment
        const int have = i0 + bi < s.cnt ? p.n - (p.tile + i0 + bi) * C::kTile - bj : 0;
        __syncwarp();
#pragma unroll
        for (int x0 = 0; x0 < kHeads; x0 += 4) {   // four heads: eight independent chains
            if (x0 >= s.heads) break;
            float y[8];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4 rc = sh.rowc[x0 + x];
                const float2 z = zn[x0 + x];
                y[2 * x] = have > 0 ? fmaxf(fmaf(phi(MODE, z.x, rc.x), rc.y, rc.z), 0.f) : 0.f;
                y[2 * x + 1] = have > 1 ? fmaxf(fmaf(phi(MODE, z.y, rc.x), rc.y, rc.z), 0.f) : 0.f;
            }
            powers(y, g.a.p);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (x0 + x < s.heads) {
                    const float2 v = make_float2(y[2 * x], y[2 * x + 1]);
                    wsum[x0 + x] += v.x + v.y;
                    wbuf[(x0 + x) * 32 + (lane ^ (x << 2))] = split_weights<T>(v);
                    if (g.a.scores && have > 0) *reinterpret_cast<float2 *>(zl + ((long long)i0 * g.sp.zg + x0 + x) * C::kTile) = v;
                }
        }
        __syncwarp();
        fetch(i0 + C::kBatch);
        const int upto = min(C::kBatch, s.cnt - i0);
        for (int i = 0; i < upto; ++i) {
            uint2 ws[C::kEights];
#pragma unroll
            for (int u = 0; u < C::kEights; ++u) {
                ws[u] = make_uint2(0u, 0u);
                if (head < s.heads) ws[u] = wbuf[head * 32 + ((i * C::kPairs + u * 4 + c4) ^ ((head & 3) << 2))];
            }
            w.stage([&](uint32_t tile) { value_tile<T, D>(tile, ws, p.n - (p.tile + i0 + i) * C::kTile, o); });
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < kHeads; ++x) {
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) wsum[x] += __shfl_xor_sync(0xffffffffu, wsum[x], e);
        if (head == x) sum = wsum[x];
    }
    // a row whose constants are NaN has weights that max() has made 0
    const bool none = isnan(sh.rowc[head].y) && head < s.heads;
    __syncwarp();
    finish_values<T, D, false>(w, p, s, 0.f, none ? NAN : sum, o);
}

// (reference, sum of w) over the row's segments i = first, first + step, ...
// of the head whose entries start at `at` (the whole warp calls it).
__device__ __forceinline__ float2 join_sums(const float2 *at, int zg, int first, int count, int step) {
    float2 x = make_float2(kLowest, 0.f);
#pragma unroll 4
    for (int i = first; i < count; i += step) x = join_pair(x, __ldcg(at + (long long)i * zg));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = join_pair(x, shuffle_xor(x, o));
    return x;
}

// An output row (query head) of many segments: the warps take every kWarps-th.
template <typename T, int D>
__device__ void join_row(const Worker<D> &w, int r) {
    constexpr int kPerLane = D / 32;
    using Vec = typename std::conditional<kPerLane == 4, float4, float2>::type;
    const Args &g = w.g;
    const PagedCache &c = g.a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = g.a.H / c.Hkv;
    Vec *part = reinterpret_cast<Vec *>(w.merge);
    const int b = r / g.a.H, hq = r % g.a.H, gq = hq % G, hr = hq / G * g.sp.blocks + gq / kHeads;
    const int n = paged_len(c, b), nt = tiles_of<D>(n);
    uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(g.a.out) + (long long)r * D + lane * kPerLane);
    const int row = b * g.sp.heads_rows + hr;
    const Segments sg = segments_of(w.chunks, row, tiles_before<D>(c, b) * g.sp.heads_rows + hr * nt, nt);
    const int count = sg.count;
    if (threadIdx.x == 0) wait_count(g.s.summed + row, (unsigned)count, &w.sh, c.err);
    compute_sync();
    const float2 *sums = g.s.sums + (long long)sg.first * g.sp.zg + gq % kHeads;
    const float *o = g.s.o + ((long long)sg.first * g.sp.zg + gq % kHeads) * D + lane * kPerLane;
    float acc[kPerLane];
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) acc[e] = 0.f;
    const float2 all = join_sums(sums, g.sp.zg, lane, count, 32);
    for (int i0 = warp; i0 < count; i0 += 32 * kWarps) {
        const int mine = i0 + lane * kWarps;
        const float f = mine < count ? ptx::ex2(__ldcg(sums + (long long)mine * g.sp.zg).x - all.x) : 0.f;
        const int cnt = min(32, (count - i0 + kWarps - 1) / kWarps);
#pragma unroll 8
        for (int i = 0; i < cnt; ++i) {
            const Vec v = __ldcg(reinterpret_cast<const Vec *>(o + (long long)(i0 + i * kWarps) * g.sp.zg * D));
            const float fi = __shfl_sync(0xffffffffu, f, i);
            acc[0] = fmaf(v.x, fi, acc[0]);
            acc[1] = fmaf(v.y, fi, acc[1]);
            if constexpr (kPerLane == 4) {
                acc[2] = fmaf(v.z, fi, acc[2]);
                acc[3] = fmaf(v.w, fi, acc[3]);
            }
        }
    }
    if constexpr (kPerLane == 4) part[warp * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    else part[warp * 32 + lane] = make_float2(acc[0], acc[1]);
    compute_sync();
    if (warp == 0) {
        for (int u = 1; u < kWarps; ++u) {
            const Vec v = part[u * 32 + lane];
            acc[0] += v.x;
            acc[1] += v.y;
            if constexpr (kPerLane == 4) {
                acc[2] += v.z;
                acc[3] += v.w;
            }
        }
        const float inv = isnan(all.x) ? NAN : 1.f / all.y;
#pragma unroll
        for (int e = 0; e < kPerLane; e += 2) out[e / 2] = Elem<T>::pack(acc[e] * inv, acc[e + 1] * inv);
    }
    compute_sync();   // before `merge` is written again
}

// The rows of sequences without tokens (zeros) and of those with a length
// outside the cache (NaN): by all CTAs.
template <typename T, int D>
__device__ void empty_rows(const Args &g) {
    const PagedCache &c = g.a.c;
    for (int b = blockIdx.x; b < c.B; b += g.sp.ctas) {
        if (paged_len(c, b)) continue;
        const float x = c.lens[b] ? NAN : 0.f;
        uint2 *out = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.a.out) + (long long)b * g.a.H * D);
        for (int i = threadIdx.x; i < g.a.H * D / 4; i += kCompute) out[i] = make_uint2(Elem<T>::pack(x, x), Elem<T>::pack(x, x));
    }
}

// The scores of a segment's tokens, by the segment of the first block of heads.
template <int D, int MODE>
__device__ void score_segment(const Worker<D> &w, const Place &p, const Segment &s) {
    using C = Config<D>;
    const Args &g = w.g;
    const PagedCache &c = g.a.c;
    Shared &sh = w.sh;
    if (s.g0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = g.a.H / c.Hkv, h = p.hr / g.sp.blocks, start = p.t - p.tile;
    compute_sync();
    if (threadIdx.x < g.sp.blocks) {
        const Segments sg = segments_of(w.chunks, s.row + (int)threadIdx.x, start + (int)threadIdx.x * p.nt, p.nt);
        if (sg.count > 1 || g.sp.blocks > 1) wait_count(g.s.summed + s.row + threadIdx.x, (unsigned)sg.count, &sh, c.err);
    }
    compute_sync();
    for (int gq = warp; gq < G; gq += kWarps) {
        const Segments sg = segments_of(w.chunks, s.row + gq / kHeads, start + gq / kHeads * p.nt, p.nt);
        const float2 x = join_sums(g.s.sums + (long long)sg.first * g.sp.zg + gq % kHeads, g.sp.zg, lane, sg.count, 32);
        if (lane == 0) sh.rowc[gq] = make_float4(x.x, isnan(x.x) ? NAN : 1.f / x.y, 0.f, 0.f);
    }
    compute_sync();
    // four slots per thread
    constexpr int kThreads = C::kTile / 4;
    const bool vec = ((reinterpret_cast<uintptr_t>(g.a.scores) | reinterpret_cast<uintptr_t>(g.a.scores_out)) & 15) == 0;
    const int slot0 = (threadIdx.x % kThreads) * 4;
    const size_t base = ((size_t)p.b * c.Hkv + h) * c.capacity();
#pragma unroll 2
    for (int i = threadIdx.x / kThreads; i < s.cnt; i += kCompute / kThreads) {
        const int slot = (p.tile + i) * C::kTile + slot0, have = p.n - slot;
        if (have <= 0) continue;
        const float *from = g.a.scores + base + slot;
        float *to = g.a.scores_out + base + slot;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), add = x;
        if (vec && have >= 4) {
            x = __ldcg(reinterpret_cast<const float4 *>(from));
        } else {
            x.x = from[0];
            if (have > 1) x.y = from[1];
            if (have > 2) x.z = from[2];
            if (have > 3) x.w = from[3];
        }
#pragma unroll 4
        for (int gq = 0; gq < G; ++gq) {
            const long long tile = start + gq / kHeads * p.nt + p.tile + i;
            float4 z = __ldcg(reinterpret_cast<const float4 *>(&g.s.z[(tile * g.sp.zg + gq % kHeads) * C::kTile + slot0]));
            const float4 rc = sh.rowc[gq];
            if (!is_reweight(MODE)) z = make_float4(phi(MODE, z.x, rc.x), phi(MODE, z.y, rc.x), phi(MODE, z.z, rc.x), phi(MODE, z.w, rc.x));
            add.x = fmaf(z.x, rc.y, add.x);
            add.y = fmaf(z.y, rc.y, add.y);
            add.z = fmaf(z.z, rc.y, add.z);
            add.w = fmaf(z.w, rc.y, add.w);
        }
        x = make_float4(x.x + add.x, x.y + add.y, x.z + add.z, x.w + add.w);
        if (vec && have >= 4) {
            *reinterpret_cast<float4 *>(to) = x;
        } else {
            to[0] = x.x;
            if (have > 1) to[1] = x.y;
            if (have > 2) to[2] = x.z;
            if (have > 3) to[3] = x.w;
        }
    }
}

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kBlock, (Config<D>::kPerSm))
paged_decode(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, const __grid_constant__ Args g) {
    using C = Config<D>;
    constexpr bool kTwoPass = is_reweight(MODE);
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const PagedCache &c = g.a.c;
    const uint32_t ring = (ptx::smem_u32(dyn) + 1023u) & ~1023u;
    float *merge = reinterpret_cast<float *>(dyn + (ring - ptx::smem_u32(dyn)) + C::kStages * C::kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // A ticket is taken only when the tiles of the item before are all on their way
    // (the ring keeps the compute warps busy meanwhile): taken earlier, some CTAs
    // would hold two large chunks while others have none.
    unsigned ticket = 0;
    auto take = [&] {
        if (lane == 0) ticket = atomicAdd(g.s.next, 1u);
    };
    if (warp == kWarps) {
        take();
        if (lane < 2) ptx::prefetch_tensormap(lane ? &vm : &km);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.empty[s]), kWarps);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.item_full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.item_empty[s]), kWarps);
        }
        sh.abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    int longest = 0;
    const int per_row = tiles_before<D>(c, c.B, &longest);
    // with a second visit to the chunks each CTA should have one, else the finer the better
    const bool revisit = kTwoPass || g.a.scores;
    const Chunks chunks(per_row * g.sp.heads_rows, g.sp.ctas, revisit);
    const int n_chunks = chunks.count();
    __syncthreads();
    if (warp == kWarps) {
        int it = 0, q = 0;
        // hands an item to the compute warps and streams its tiles
        auto post = [&](int kind, int index) {
            Item x = {};
            x.kind = kind;
            x.index = index;
            if (kind < kJoinRow) {
                x.p = locate<D>(c, g.sp.heads_rows, chunks.begin(index));
                x.t1 = chunks.end(index);
            }
            if (q > 1 && !__all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh.item_empty[q & 1]), ((q >> 1) - 1) & 1, &sh, c.err, kErrItem, true)))
                return false;
            if (lane == 0) {
                sh.item[q & 1] = x;
                ptx::mbar_arrive(ptx::smem_u32(&sh.item_full[q & 1]));
            }
            ++q;
            __syncwarp();
            if (kind == kScoreTiles) return produce<D, 0>(g, &km, &vm, &sh, ring, x.p, x.t1, it);
            if (kind == kValueTiles) return produce<D, kTwoPass ? 1 : 2>(g, &km, &vm, &sh, ring, x.p, x.t1, it);
            return true;
        };
        bool go = true;
        int mine = 0;
        int i = (int)__shfl_sync(0xffffffffu, ticket, 0);
        while (go && i < n_chunks) {
            if (revisit) {
                if (lane == 0) sh.mine[mine] = (unsigned short)i;
                ++mine;
            }
            go = post(kTwoPass ? kScoreTiles : kValueTiles, i);
            take();
            i = (int)__shfl_sync(0xffffffffu, ticket, 0);
        }
        __syncwarp();
        if (kTwoPass)
            for (int k = 0; go && k < mine; ++k) go = post(kValueTiles, sh.mine[k]);
        // query heads of rows of many segments
        if (longest > (kFewSegments - 1) * chunks.small)
            for (int r = blockIdx.x; go && r < c.B * g.a.H; r += g.sp.ctas) {
                const int G = g.a.H / c.Hkv, b = r / g.a.H, hq = r % g.a.H, hr = hq / G * g.sp.blocks + hq % G / kHeads;
                const int nt = tiles_of<D>(paged_len(c, b));
                if (nt > 0 && segments_of(chunks, 0, tiles_before<D>(c, b) * g.sp.heads_rows + hr * nt, nt).count > kFewSegments) go = post(kJoinRow, r);
            }
        if (g.a.scores)
            for (int k = 0; go && k < mine; ++k) go = post(kAddScores, sh.mine[k]);
        if (go) post(kEnd, 0);
        // the last copies have landed before the CTA ends
        if (lane == 0)
            for (int k = max(0, it - C::kStages); k < it; ++k)
                bounded_wait(ptx::smem_u32(&sh.full[k % C::kStages]), (k / C::kStages) & 1, &sh, c.err, kErrDrain, false);
        __syncwarp();
        return;
    }
    empty_rows<T, D>(g);
    Worker<D> w{g, sh, ring, merge, chunks};
    for (int q = 0;; ++q) {
        if (!__all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh.item_full[q & 1]), (q >> 1) & 1, &sh, c.err, kErrItem, true))) break;
        const Item x = sh.item[q & 1];
        if (x.kind == kEnd) break;
        if (x.kind == kJoinRow) {
            join_row<T, D>(w, x.index);
        } else {
            Place p = x.p;
            while (p.t < x.t1) {
                const Segment s = segment_at(g, chunks, p, x.t1);
                w.bad = false;
                if (x.kind == kAddScores) {
                    score_segment<D, MODE>(w, p, s);
                } else if constexpr (kTwoPass) {
                    if (x.kind == kScoreTiles) scores_segment<T, D, MODE>(w, p, s, x.t1);
                    else values_segment<T, D, MODE>(w, p, s);
                } else {
                    one_pass_segment<T, D, MODE>(w, p, s, x.t1);
                }
                p.t += s.cnt;
                if (p.t < x.t1) next_row<D>(c, g.sp.heads_rows, p);
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.item_empty[q & 1]));
    }
}

// CTAs of an instance that fit the current device at once (also sets its
// shared-memory attribute).
template <typename T, int D, int MODE>
cudaError_t resident(int *ctas) {
    static PerDeviceOnce once;
    return per_device_once(once, ctas, [](int &v) {
        int sms = 0, per_sm = 0;
        cudaError_t e = device_sms(&sms);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_decode<T, D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Config<D>::kSmem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, paged_decode<T, D, MODE>, kBlock, Config<D>::kSmem);
        v = sms * per_sm;
        return e;
    });
}

template <typename T, int D, int MODE>
cudaError_t launch_mode(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, cudaStream_t stream) {
    void *args[] = {(void *)&km, (void *)&vm, (void *)&g};
    return cudaLaunchKernel((const void *)paged_decode<T, D, MODE>, dim3(g.sp.ctas), dim3(kBlock), args, (size_t)Config<D>::kSmem, stream);
}

// One call per (type, d) and file, so that the instances compile in parallel.
#define LSSAR_PAGED_DECODE_INSTANCES(T, D, NAME)                                                                            \
    cudaError_t NAME##_resident(int mode, int *ctas) {                                                                      \
        switch (mode) {                                                                                                     \
            case kSoftmax: return resident<T, D, kSoftmax>(ctas);                                                           \
            case kLssa: return resident<T, D, kLssa>(ctas);                                                                 \
            case kLssar: return resident<T, D, kLssar>(ctas);                                                               \
            case kSoftmaxRw: return resident<T, D, kSoftmaxRw>(ctas);                                                       \
            default: return resident<T, D, kSigmoidRw>(ctas);                                                               \
        }                                                                                                                   \
    }                                                                                                                       \
    cudaError_t NAME##_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, cudaStream_t stream) {           \
        switch (g.a.mode) {                                                                                                 \
            case kSoftmax: return launch_mode<T, D, kSoftmax>(km, vm, g, stream);                                           \
            case kLssa: return launch_mode<T, D, kLssa>(km, vm, g, stream);                                                 \
            case kLssar: return launch_mode<T, D, kLssar>(km, vm, g, stream);                                               \
            case kSoftmaxRw: return launch_mode<T, D, kSoftmaxRw>(km, vm, g, stream);                                       \
            default: return launch_mode<T, D, kSigmoidRw>(km, vm, g, stream);                                               \
        }                                                                                                                   \
    }

cudaError_t bf16_d64_resident(int mode, int *ctas);
cudaError_t bf16_d128_resident(int mode, int *ctas);
cudaError_t fp16_d64_resident(int mode, int *ctas);
cudaError_t fp16_d128_resident(int mode, int *ctas);
cudaError_t bf16_d64_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, cudaStream_t stream);
cudaError_t bf16_d128_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, cudaStream_t stream);
cudaError_t fp16_d64_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, cudaStream_t stream);
cudaError_t fp16_d128_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, cudaStream_t stream);

}  // namespace paged
}  // namespace lssar
