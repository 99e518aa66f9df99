// Paged cache, decode: one new query row per head against a sequence's pages,
// in every mode of the forward (row i = the sequence's length), grouped heads,
// and the attention weight that each cached token receives added up.
//
// Mathematics, per (sequence b, query head): z_j = the score in log2 units,
// phi_j = the mode's normaliser, S1 = sum phi_j, m = max z_j; the weights are
// w_j = phi_j (softmax: 2^(z_j - m)), or with re-weighting max(kappa (phi_j -
// theta), 0)^p with kappa, theta from S1, m and i; out = sum w_j v_j / sum w_j.
//
// What bounds it: every key and value row is read once from HBM, 4d bytes per
// (token, key head) against 4Gd flops for a group of G query heads, while G <= 8; each
// further block of 8 query heads reads them again (from L2 where they are still there).
// Measured: 8 sequences of 16K tokens, 12 heads of 64, with scores 82 us; 480 MB of ragged
// grouped sequences, one pass, 86 us (5.6 TB/s; the copies alone reach 6.06).
//
// Split.  The tokens of all sequences are cut into tiles of 16 KB of one key
// head, numbered through (sequence, key head, block of 8 query heads, tile); each
// CTA takes an equal run of tiles wherever rows begin or end, so that lengths
// of any mix load the SMs evenly.  The part of a row inside one run is a segment.
// The lengths are on the device: each warp finds its run by a prefix sum.
//   softmax, LSSA: paged_stream<kBoth>   one pass over K and V tiles, weights
//                  relative to a running maximum;
//   re-weighting:  paged_stream<kScores> K tiles -> z (scratch), (m, S1) per segment,
//                  paged_stream<kValues> row constants from all of the row's
//                  segments, z -> w, V tiles (asked for before the scores are in,
//                  as soon as CTAs of the scores kernel make room);
//   then           paged_join            sums the segments of each row, and adds
//                  each token's normalised weights to its score.
// Each kernel is a programmatic dependent of the one before it.  (One kernel for
// all, with per-row counts between its passes, took as long: its 140 KB of code
// were fetched cold at each step.  Warps that work alone, with a ring each, took
// 20 to 40 % longer: a tile's copies and look-ups cost more than its arithmetic.)
//
// Products on mma.sync m16n8k16: a decode row has G <= 8 query heads per key head
// in a block, which a 128-row tcgen05 tile would leave almost empty, and the
// tensor work is a small part of the time that HBM needs.  The 16 rows of an
// operand carry the 8 heads and, for free, something else that is needed:
//   scores: rows 8-15 the queries, rows 0-7 the tile's own 8 keys, so that one
//           product gives q.k and, on the diagonal, |k|^2;
//   values: rows 8-15 the weights rounded to 16 bits, rows 0-7 what the rounding
//           left over, so that weights keep 16 bits (fp16: and 2^-37 of the largest).
// K and V tiles come by TMA (128-byte swizzle), a piece of a page at a time.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"
#include "row_weights.cuh"
#include "tc_host.cuh"
#include "tc_ptx.cuh"

namespace lssar {
namespace paged {

enum Phase : int { kScores = 0, kValues = 1, kBoth = 2 };

constexpr int kWarps = 4;                     // compute warps, each a quarter of every tile's keys
constexpr int kCompute = kWarps * 32;
constexpr int kBlock = kCompute + 32;         // + the producer warp
constexpr int kHeads = 8;                     // query heads per block of heads
constexpr int kMaxGroup = 128;                // H / Hkv
constexpr float kLowest = -3.0e38f;           // below every score, and finite
constexpr uint64_t kWaitLimitNs = 2000000000ull;
enum : unsigned { kErrFull = 53, kErrEmpty, kErrDrain };

__host__ __device__ constexpr int tile_keys(int d) { return 8192 / d; }   // 16 KB of K or V

template <int D, int PHASE>
struct Config {
    static constexpr int kTile = tile_keys(D);
    static constexpr int kKeys = kTile / kWarps;       // keys per warp and tile
    static constexpr int kEights = kKeys / 8;          // blocks of 8 keys
    static constexpr int kPairs = kKeys / 2;           // pairs of keys per warp and tile
    static constexpr int kBatch = 32 / kPairs;         // tiles whose weights are formed together (32 pairs)
    static constexpr int kStageBytes = kTile * D * 2;
    // CTAs per SM and stages of each.  d = 64: 3 x 3 (3 x 2 as fast, 2 x 5 4 % slower on
    // 8 x 16K).  d = 128: 2 x 4; three CTAs leave 128 registers a thread, too few for the
    // one-pass kernel: 104 against 91 us on a ragged batch of 480 MB, 43 against 39 us on
    // 64 short sequences.
    static constexpr int kStages = D == 64 ? 3 : 4;
    static constexpr int kPerSm = D == 64 ? 3 : 2;
    static constexpr int kMerge = PHASE == kScores ? 0 : kWarps * kHeads * D * 4;   // the warps' sums of w v
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kMerge;
};

// How a launch is laid out.
struct Split {
    int G;                 // H / Hkv
    int blocks;            // blocks of kHeads query heads per key head
    int heads_rows;        // Hkv * blocks: rows per sequence
    int zg;                // heads stored per tile: min(G, kHeads)
    int ctas;              // CTAs that share the tiles
};

struct Scratch {
    float *z;              // [tile][zg][keys]: z, then w (re-weighting with scores)
    float2 *stats;         // [segment][zg]: max of z, sum of phi
    float2 *sums;          // [segment][zg]: reference of the exponent (softmax, LSSA), sum of w
    float *o;              // [segment][zg][D]: sum of w v
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
    int b, h, nb, tile;    // sequence, key head, block of query heads, tile of the row
    int n, nt;             // length and tiles of the sequence
};

template <int D>
__device__ __forceinline__ int tiles_of(int n) {
    return (n + tile_keys(D) - 1) / tile_keys(D);
}

// Lengths as they are used: 0 where they are outside the cache.  (Those of many
// sequences are asked for at once; the error word is written after them.)
__device__ __forceinline__ int usable(int n, int capacity) { return (unsigned)n <= (unsigned)capacity ? n : 0; }

// Tiles of sequences [0, upto) for one row of each (the whole warp calls it).
template <int D>
__device__ __forceinline__ int tiles_before(const PagedCache &c, int upto) {
    const int cap = c.capacity();
    int x = 0;
    bool bad = false;
#pragma unroll 4
    for (int b = threadIdx.x & 31; b < upto; b += 32) {
        const int n = c.lens[b];
        bad |= usable(n, cap) != n;
        x += tiles_of<D>(usable(n, cap));
    }
    if (bad) atomicCAS(c.err, 0u, (unsigned)kErrPagedLength);
    return __reduce_add_sync(0xffffffffu, x);
}

// The place of tile t < total (the whole warp calls it): eight sequences per lane.
template <int D>
__device__ __noinline__ Place locate(const PagedCache &c, int blocks, int t) {
    const int lane = threadIdx.x & 31, rows_per_seq = c.Hkv * blocks, cap = c.capacity();
    Place p;
    int before = 0;
#pragma unroll 1
    for (int b0 = lane * 8;; b0 += 256) {
        int n[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = b0 + j < c.B ? c.lens[b0 + j] : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            n[j] = usable(n[j], cap);
            sum += tiles_of<D>(n[j]);
        }
        int end = sum * rows_per_seq;
        const int own = end;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + end > t);
        if (hit) {
            int in = t - (before + end - own), at = 0, len = 0;
            bool found = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int tiles = tiles_of<D>(n[j]) * rows_per_seq;
                if (!found && in < tiles) {
                    found = true;
                    at = b0 + j;
                    len = n[j];
                }
                if (!found) in -= tiles;
            }
            const int l = __ffs(hit) - 1;
            in = __shfl_sync(0xffffffffu, in, l);
            p.b = __shfl_sync(0xffffffffu, at, l);
            p.n = __shfl_sync(0xffffffffu, len, l);
            p.nt = tiles_of<D>(p.n);
            const int hr = in / p.nt;
            p.tile = in - hr * p.nt;
            p.h = hr / blocks;
            p.nb = hr - p.h * blocks;
            p.t = t;
            return p;
        }
        before += __shfl_sync(0xffffffffu, end, 31);
    }
}

// On to the first tile of the next row that has one.
template <int D>
__device__ __forceinline__ void next_row(const PagedCache &c, int blocks, Place &p) {
    p.tile = 0;
    if (++p.nb < blocks) return;
    p.nb = 0;
    if (++p.h < c.Hkv) return;
    p.h = 0;
#pragma unroll 1
    do {
        if (++p.b >= c.B) return;
        p.n = paged_len(c, p.b);
        p.nt = tiles_of<D>(p.n);
    } while (p.nt == 0);
}

// The element types as operands.  A weight is two of them, rounded and the remainder.  fp16
// has no step below 2^-24: weights relative to the row's largest one would lose what is
// below 2^-25 of it, which many keys together make count, so that the largest ones are
// put between 2^13 and 2^15 (at most 1.45 2^15 = 47514 in LSSA), where the least step is
// 2^-37 of them and 2^24 keys lose 2^-14.  bf16 has fp32's range.
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static constexpr float kRoom = 0.f, kLag = 8.f;   // one pass: log2 of the largest weight is in kRoom + [0, kLag]
    static constexpr float kTop = 1.f;                // re-weighting: the largest weight
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
    static constexpr float kRoom = 13.f, kLag = 2.f;
    static constexpr float kTop = 32768.f;
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
    return tile + (chunk >> 3) * (tile_keys(D) * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory"); }

struct Shared {
    uint64_t full[4], empty[4];
    int bad[4];                     // the stage's tile names a page that is none
    float2 red[kWarps][kHeads];
    float4 rowc[kHeads];             // RowConstants
    int abort_flag;
};

// (Inline all the same: a call would save the accumulators.)
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, Shared *sh, unsigned *err, unsigned code, bool honour_abort) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
#pragma unroll 1
    while (!ptx::mbar_try_wait_sleep(bar, parity, 100000)) {
        if (honour_abort && *(volatile int *)&sh->abort_flag) return false;
        if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicCAS(err, 0u, code);
            *(volatile int *)&sh->abort_flag = 1;
            return false;
        }
    }
    return true;
}

// The segments of the row that starts at tile `start`: `count` of them, with
// scratch entries first, first + 1, ... = row + CTA (both grow along the
// numbering, so that no two segments share one).
struct Segments {
    int first, count;
};
__device__ __forceinline__ Segments segments_of(int row, int start, int nt, int run) {
    const int a = start / run;
    return Segments{row + a, (start + nt - 1) / run - a + 1};
}

// For the debug build's checks: entries of the segments' scratch; whether the `cnt` tiles
// from p on are tiles of one row and of the scratch.
__device__ __forceinline__ int segments_of_all(const Args &g) { return g.a.c.B * g.sp.heads_rows + g.sp.ctas; }
template <int D>
__device__ __forceinline__ bool in_numbering(const Args &g, const Place &p, int cnt) {
    const PagedCache &c = g.a.c;
    return p.b >= 0 && p.b < c.B && p.h >= 0 && p.h < c.Hkv && p.n <= c.capacity() && p.tile >= 0 && cnt > 0 && p.tile + cnt <= p.nt &&
           p.t >= 0 && p.t + cnt <= c.B * g.sp.heads_rows * tiles_of<D>(c.capacity());
}

// (m, s): sums s relative to 2^m.  A row that must not be used has s = NaN.
__device__ __forceinline__ float2 join_pair(float2 x, float2 y) {
    const float m = fmaxf(x.x, y.x);
    return make_float2(m, x.y * ptx::ex2(x.x - m) + y.y * ptx::ex2(y.x - m));
}
// ... or, not RELATIVE, a maximum and a plain sum.
template <bool RELATIVE>
__device__ __forceinline__ float2 join(float2 x, float2 y) {
    return RELATIVE ? join_pair(x, y) : make_float2(fmaxf(x.x, y.x), x.y + y.y);
}
__device__ __forceinline__ float2 shuffle_xor(float2 x, int o) {
    return make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o));
}

// The weights of two scores in the one-pass modes, relative to 2^ref: 2^(z - ref), or
// log2(1 + 2^z) 2^-ref with lift = 2^-ref.
template <int MODE>
__device__ __forceinline__ float2 weights(float2 z, float ref, float lift) {
    const float2 w = phi(MODE, z, ref);
    return MODE == kSoftmax ? w : make_float2(w.x * lift, w.y * lift);
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

// Producer warp: the tiles of the CTA's run, in order, through the ring.
template <int D, int PHASE>
__device__ __forceinline__ void produce(const Args &g, const CUtensorMap *km, const CUtensorMap *vm, Shared *sh, uint32_t ring, Place p, int t1) {
    using C = Config<D, PHASE>;
    const PagedCache &c = g.a.c;
    const int lane = threadIdx.x & 31, piece_rows = g.piece_rows, ps = c.page_size;
    const bool mine = lane * piece_rows < C::kTile;
    const uint32_t dst0 = ring + lane * piece_rows * 128;
    // the page and row of this lane's piece of the next tile; -1: past the row's end, -2: none of the pool
    int pg = -1, row = 0;
    auto look_up = [&] {
        const int s0 = p.tile * C::kTile + lane * piece_rows, i = s0 / ps;
        pg = -1;
        if (!mine || s0 >= p.n) return;
        row = p.h * ps + s0 - i * ps;
        pg = paged_page(c, p.b, i);
        if (pg < 0) pg = -2;
    };
    int slot = 0, lap = 0, used = 0;
    look_up();
#pragma unroll 1
    while (true) {
        const unsigned ok = __ballot_sync(0xffffffffu, pg >= 0), bad = __ballot_sync(0xffffffffu, pg == -2);
        const int page = pg, y = row;
        // the next tile's pages are looked up while this one waits for its stage
        const bool more = ++p.t < t1;
        if (more) {
            if (++p.tile == p.nt) {
                next_row<D>(c, g.sp.blocks, p);
                // the compute warps will want that row's queries soon (64 short sequences:
                // 39.3 -> 38.1 us, a ragged batch 91 -> 87)
                if (PHASE != kValues && lane < min(kHeads, g.sp.G - p.nb * kHeads) * (D / 64)) {
                    const uint16_t *q = static_cast<const uint16_t *>(g.a.q) + p.b * g.a.q_b + (p.h * g.sp.G + p.nb * kHeads + lane / (D / 64)) * g.a.q_h;
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(q + lane % (D / 64) * 64));
                }
            }
            look_up();
        }
#pragma unroll 1
        for (int u = 0; u < (PHASE == kBoth ? 2 : 1); ++u) {
            if (lap > 0 && !__all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh->empty[slot]), (lap - 1) & 1, sh, c.err, kErrEmpty, true))) goto out;
            const uint32_t full = ptx::smem_u32(&sh->full[slot]), dst = dst0 + slot * C::kStageBytes;
            const CUtensorMap *map = PHASE == kValues || u == 1 ? vm : km;
            if (lane == 0) {
                sh->bad[slot] = bad != 0;
                ptx::mbar_arrive_expect_tx(full, (uint32_t)__popc(ok) * piece_rows * D * 2);
            }
            __syncwarp();
            if (page >= 0 && dcheck(y >= 0 && y + piece_rows <= c.Hkv * ps && page < c.n_pages && mine, c.err, kDbgTma)) {
                ptx::tma_load_3d(dst, map, full, 0, y, page);
                if (D == 128) ptx::tma_load_3d(dst + C::kTile * 128, map, full, 64, y, page);
            }
            ++used;
            if (++slot == C::kStages) {
                slot = 0;
                ++lap;
            }
        }
        if (!more) break;
    }
out:
    // the last copies have landed before the CTA ends
    if (lane == 0)
        for (int i = max(0, used - C::kStages); i < used; ++i)
            bounded_wait(ptx::smem_u32(&sh->full[i % C::kStages]), (i / C::kStages) & 1, sh, c.err, kErrDrain, false);
    __syncwarp();
}

// The scores z of the warp's keys of a tile (blocks of 8 keys): head lane / 4,
// keys 2 (lane % 4) + {0, 1} of each block.
template <typename T, int D, bool RAW>
__device__ __forceinline__ void score_tile(uint32_t tile, const uint32_t (&qf)[D / 16][2], float scale, float2 (&z)[Config<D, kScores>::kEights]) {
    using C = Config<D, kScores>;
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
            z[u].x *= ptx::rsqrt(fmaxf(ka, 1e-24f));   // |k| clamped at 1e-12 as everywhere
            z[u].y *= ptx::rsqrt(fmaxf(kb, 1e-24f));
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
__device__ __forceinline__ void value_tile(uint32_t tile, const uint2 (&w)[Config<D, kValues>::kEights], int left, float (&o)[D / 8][4]) {
    using C = Config<D, kValues>;
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

template <typename T, int D, int MODE, int PHASE>
__global__ void __launch_bounds__(kBlock, (Config<D, PHASE>::kPerSm))
paged_stream(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, const __grid_constant__ Args g) {
    using C = Config<D, PHASE>;
    constexpr bool kRaw = MODE == kSoftmax || MODE == kSoftmaxRw;
    constexpr bool kRelative = PHASE == kScores ? kRaw : PHASE == kBoth;   // sums relative to 2^reference
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    const PagedCache &c = g.a.c;
    const uint32_t ring = (ptx::smem_u32(dyn) + 1023u) & ~1023u;
    float *merge = reinterpret_cast<float *>(dyn + (ring - ptx::smem_u32(dyn)) + C::kStages * C::kStageBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::launch_dependents();
    if (threadIdx.x == kCompute) {   // the producer's first lane
        ptx::prefetch_tensormap(PHASE == kValues ? &vm : &km);
        if (PHASE == kBoth) ptx::prefetch_tensormap(&vm);
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.empty[s]), kWarps);
        }
        sh.abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    const int total = tiles_before<D>(c, c.B) * g.sp.heads_rows, run = max(1, (total + g.sp.ctas - 1) / g.sp.ctas);
    const int t0 = blockIdx.x * run, t1 = min(t0 + run, total);
    __syncthreads();
    if (t0 >= total) {
        if (PHASE == kValues) ptx::grid_dependency_wait();   // this grid ends after the one before it
        return;
    }
    Place p = locate<D>(c, g.sp.blocks, t0);
    if (warp == kWarps) {
        produce<D, PHASE>(g, &km, &vm, &sh, ring, p, t1);
        return;
    }
    if (PHASE == kValues) ptx::grid_dependency_wait();   // z and the segments' statistics
    const int head = lane >> 2, c4 = lane & 3;
    int slot = 0, parity = 0;
    bool bad = false;
    // waits for the next stage and uses it
    auto stage = [&](auto &&use) {
        const bool ok = __all_sync(0xffffffffu, bounded_wait(ptx::smem_u32(&sh.full[slot]), parity, &sh, c.err, kErrFull, true));
        bad |= !ok || sh.bad[slot];
        use(ring + slot * C::kStageBytes);
        __syncwarp();
        if (lane == 0 && ok) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[slot]));
        if (++slot == C::kStages) {
            slot = 0;
            parity ^= 1;
        }
    };
#pragma unroll 1
    while (true) {   // one segment per turn
        const int row = p.b * g.sp.heads_rows + p.h * g.sp.blocks + p.nb;
        const Segments sg = segments_of(row, p.t - p.tile, p.nt, run);
        const int seg = row + blockIdx.x, g0 = p.nb * kHeads, heads = min(kHeads, g.sp.G - g0), cnt = min(t1 - p.t, p.nt - p.tile);
        const bool mine = head < heads;
        // (every index of the scratch and the outputs follows from these)
        if (!dcheck(in_numbering<D>(g, p, cnt) && heads > 0 && p.nb < g.sp.blocks && sg.first + sg.count <= segments_of_all(g) && seg < segments_of_all(g), c.err, kDbgItem)) break;
        bad = false;
        float2 st = make_float2(PHASE == kValues ? 0.f : kLowest, 0.f);   // (maximum or reference, sum of phi or w)
        float lift = 0.f;   // LSSA: 2^-reference
        float o[PHASE == kScores ? 1 : D / 8][4];
        if constexpr (PHASE != kScores) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        }
        if constexpr (PHASE == kValues) {
            // Weights of kBatch tiles at a time, in pairs of keys spread over all lanes
            // whatever the number of heads, and to the operand layout through shared
            // memory (the warp's own part of `merge`; the place of a pair is permuted by
            // the head so that the operand reads hit every bank once).
            uint2 *wbuf = reinterpret_cast<uint2 *>(merge + warp * kHeads * D);
            const int bi = lane / C::kPairs, bj = C::kKeys * warp + 2 * (lane % C::kPairs);   // tile of the batch, first key
            float *zl = g.s.z + (long long)(p.t + bi) * g.sp.zg * C::kTile + bj;
            float2 zn[4];       // four heads of a batch, asked for one round ahead
            auto fetch = [&](int i0, int x0) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (x0 + x < heads && i0 + bi < cnt) zn[x] = __ldcg(reinterpret_cast<const float2 *>(zl + (i0 * g.sp.zg + x0 + x) * C::kTile));
            };
            fetch(0, 0);
            {   // the row's constants: 16 threads per head over its segments
                float2 x = make_float2(kLowest, 0.f);
                const int hh = threadIdx.x % kHeads;
                const float2 *at = g.s.stats + (long long)sg.first * g.sp.zg + hh;
                if (hh < heads)
#pragma unroll 4
                    for (int i = threadIdx.x / kHeads; i < sg.count; i += kCompute / kHeads) x = join<kRaw>(x, __ldcg(at + (long long)i * g.sp.zg));
                x = join<kRaw>(x, shuffle_xor(x, 8));
                x = join<kRaw>(x, shuffle_xor(x, 16));
                compute_sync();
                if (lane < kHeads) sh.red[warp][lane] = x;
                compute_sync();
                if (threadIdx.x < kHeads) {
                    x = sh.red[0][threadIdx.x];
#pragma unroll 1
                    for (int u = 1; u < kWarps; ++u) x = join<kRaw>(x, sh.red[u][threadIdx.x]);
                    const RowConstants rc = row_constants(MODE, p.n, x);
                    sh.rowc[threadIdx.x] = make_float4(rc.x, rc.kappa, rc.beta, rc.theta);
                }
                compute_sync();
            }
            float wsum[2][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) wsum[0][x] = wsum[1][x] = 0.f;
#pragma unroll 1
            for (int i0 = 0; i0 < cnt; i0 += C::kBatch) {
                // keys of the row from the lane's first on; none in a tile past the segment
                const int have = i0 + bi < cnt ? p.n - (p.tile + i0 + bi) * C::kTile - bj : 0;
                __syncwarp();
#pragma unroll 1
                for (int x0 = 0; x0 < heads; x0 += 4) {   // four heads: eight independent chains
                    float y[8];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float4 r4 = sh.rowc[x0 + x];
                        const RowConstants rc = {r4.x, r4.y, r4.z, r4.w};
                        const float2 v = above_offset(MODE, zn[x], rc);
                        y[2 * x] = have > 0 ? v.x : 0.f;
                        y[2 * x + 1] = have > 1 ? v.y : 0.f;
                    }
                    powers(y, g.a.p);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (x0 + x < heads) {
                            const float2 v = make_float2(y[2 * x], y[2 * x + 1]);
                            wsum[0][x] += x0 ? 0.f : v.x + v.y;
                            wsum[1][x] += x0 ? v.x + v.y : 0.f;
                            wbuf[(x0 + x) * 32 + (lane ^ (x << 2))] = split_weights<T>(make_float2(v.x * Elem<T>::kTop, v.y * Elem<T>::kTop));
                            if (g.a.scores && have > 0) *reinterpret_cast<float2 *>(zl + (i0 * g.sp.zg + x0 + x) * C::kTile) = v;
                        }
                    if (x0 + 4 < heads) fetch(i0, x0 + 4);
                    else fetch(i0 + C::kBatch, 0);
                }
                __syncwarp();
                const int upto = min(C::kBatch, cnt - i0);
#pragma unroll 1
                for (int i = 0; i < upto; ++i) {
                    uint2 ws[C::kEights];
#pragma unroll
                    for (int u = 0; u < C::kEights; ++u) {
                        ws[u] = make_uint2(0u, 0u);
                        if (mine) ws[u] = wbuf[head * 32 + ((i * C::kPairs + u * 4 + c4) ^ ((head & 3) << 2))];
                    }
                    stage([&](uint32_t tile) { value_tile<T, D>(tile, ws, p.n - (p.tile + i0 + i) * C::kTile, o); });
                }
            }
            // to the lanes of each head
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                // heads x and x + 4 at once: the lower half of the warp sums one, the upper the other
                const float keep = lane & 16 ? wsum[1][x] : wsum[0][x], give = lane & 16 ? wsum[0][x] : wsum[1][x];
                float v = keep + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
                for (int e = 8; e > 0; e >>= 1) v += __shfl_xor_sync(0xffffffffu, v, e);
                if ((head & 3) == x) st.y = v;   // lanes of heads 0-3 are the lower half
            }
            if (mine && isnan(sh.rowc[head].y)) st.y = NAN;   // max() has made its weights 0
        } else {
            // queries (rows past the block's heads are zero) and the row's factor
            uint32_t qf[D / 16][2];
            const uint16_t *q = static_cast<const uint16_t *>(g.a.q) + p.b * g.a.q_b + (p.h * g.sp.G + g0 + head) * g.a.q_h + 2 * c4;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int u = 0; u < 2; ++u) qf[kk][u] = mine ? *reinterpret_cast<const uint32_t *>(q + 16 * kk + 8 * u) : 0u;
            constexpr float kLog2e = 1.4426950408889634f;
            float scale = kLog2e * (D == 64 ? 0.125f : 0.08838834764831845f);   // / sqrt(D)
            if constexpr (!kRaw) {
                float ss = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float2 x = Elem<T>::unpack(qf[kk][u]);
                        ss = fmaf(x.x, x.x, ss);
                        ss = fmaf(x.y, x.y, ss);
                    }
                ss += __shfl_xor_sync(0xffffffffu, ss, 1);
                ss += __shfl_xor_sync(0xffffffffu, ss, 2);
                ss = fmaxf(ss, 1e-24f);   // |q| clamped at 1e-12
                float inv = ptx::rsqrt(ss);
                inv = inv * fmaf(-0.5f * ss * inv, inv, 1.5f);   // a Newton step: the factor multiplies every score
                scale = kLog2e * (D == 64 ? 4.1588830833596715f : 4.852030263919617f) * logf((float)p.n) * inv;   // ln D ln n / |q|
            }
            float *zrow = mine && (PHASE == kScores || g.a.scores) ? g.s.z + ((long long)p.t * g.sp.zg + head) * C::kTile + C::kKeys * warp + 2 * c4 : nullptr;
#pragma unroll 1
            for (int i = 0; i < cnt; ++i) {
                const int left = p.n - (p.tile + i) * C::kTile;
                float2 z[C::kEights];
                stage([&](uint32_t tile) { score_tile<T, D, kRaw>(tile, qf, scale, z); });
                if (left < C::kTile) {
                    const int j = C::kKeys * warp + 2 * c4;
#pragma unroll
                    for (int u = 0; u < C::kEights; ++u) {
                        if (j + 8 * u >= left) z[u].x = -INFINITY;
                        if (j + 8 * u + 1 >= left) z[u].y = -INFINITY;
                    }
                }
                if (zrow) {
#pragma unroll
                    for (int u = 0; u < C::kEights; ++u) *reinterpret_cast<float2 *>(zrow + 8 * u) = z[u];
                    zrow += g.sp.zg * C::kTile;
                }
                float top = fmaxf(z[0].x, z[0].y);
#pragma unroll
                for (int u = 1; u < C::kEights; ++u) top = fmaxf(top, fmaxf(z[u].x, z[u].y));
                if constexpr (PHASE == kScores) {
                    top = fmaxf(top, st.x);
                    if (kRaw) st.y *= ptx::ex2(st.x - top);
                    st.x = top;
#pragma unroll
                    for (int u = 0; u < C::kEights; ++u) {
                        const float2 f = phi(MODE, z[u], top);
                        st.y += f.x + f.y;
                    }
                } else {
                    // weights relative to 2^reference: m (softmax), or min(m, 0) (LSSA, whose weights
                    // are about 2^z there: 16 bits would lose them; in fp16 log2(1 + m) above 0, so
                    // that the largest weight is about 1 here too), less kRoom.  The reference
                    // follows the maximum only when that has grown by more than kLag, so that
                    // rescaling is rare and weights stay below 2^(kRoom + kLag) (LSSA: 1.45 times that;
                    // in bf16 118 times).
                    constexpr float kRoom = Elem<T>::kRoom, kMost = kRoom + Elem<T>::kLag;
                    if (MODE != kSoftmax) top = kRoom == 0.f ? fminf(top, 0.f) : top < 0.f ? top : ptx::lg2(1.f + top);
                    if (__any_sync(0xffffffffu, top - st.x > kMost)) {
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        if (kRoom != 0.f) {
                            float ref = top - kRoom;
                            if (top - ref > kMost) ref = top;            // steps of a top past 2^24
                            if (MODE != kSoftmax) ref = fmaxf(ref, -126.f);   // 2^-ref is finite
                            top = ref;
                        }
                        top = fmaxf(top, st.x);
                        const float f = ptx::ex2(st.x - top);
                        st = make_float2(top, st.y * f);
                        if (MODE != kSoftmax) lift = top > kLowest ? ptx::ex2(-top) : 0.f;
#pragma unroll
                        for (int k = 0; k < D / 8; ++k)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[k][e] *= f;
                    }
                    uint2 ws[C::kEights];
#pragma unroll
                    for (int u = 0; u < C::kEights; ++u) {
                        const float2 y = weights<MODE>(z[u], st.x, lift);
                        st.y += y.x + y.y;
                        ws[u] = split_weights<T>(y);
                    }
                    stage([&](uint32_t tile) { value_tile<T, D>(tile, ws, left, o); });
                }
            }
            // the four lanes of a head (they share the reference in the one-pass modes)
            st = join<PHASE == kScores && kRaw>(st, shuffle_xor(st, 1));
            st = join<PHASE == kScores && kRaw>(st, shuffle_xor(st, 2));
        }
        // the segment's statistics and sums over the warps
        compute_sync();
        if (c4 == 0) sh.red[warp][head] = make_float2(st.x, bad ? NAN : st.y);
        compute_sync();
        float2 all = sh.red[0][head];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) all = join<kRelative>(all, sh.red[w][head]);
        if (warp == 0 && c4 == 0 && mine) (PHASE == kScores ? g.s.stats : g.s.sums)[(long long)seg * g.sp.zg + head] = all;
        if constexpr (PHASE != kScores) {
            // a row with this segment alone is written out, the others go to scratch
            const bool whole = sg.count == 1;
            float f = kRelative ? ptx::ex2(st.x - all.x) : 1.f / Elem<T>::kTop;
            if (whole) f *= ptx::rcp(all.y);
#pragma unroll
            for (int k = 0; k < D / 8; ++k)
                *reinterpret_cast<float2 *>(&merge[(warp * kHeads + head) * D + 8 * k + 2 * c4]) =
                    make_float2((o[k][0] + o[k][2]) * f, (o[k][1] + o[k][3]) * f);
            compute_sync();
            uint16_t *out = static_cast<uint16_t *>(g.a.out) + ((long long)p.b * g.a.H + p.h * g.sp.G + g0) * D;
#pragma unroll 1
            for (int i = threadIdx.x; i < heads * D / 4; i += kCompute) {
                float4 x = reinterpret_cast<const float4 *>(merge)[i];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 y = reinterpret_cast<const float4 *>(merge)[w * kHeads * D / 4 + i];
                    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                }
                if (whole) reinterpret_cast<uint2 *>(out)[i] = make_uint2(Elem<T>::pack(x.x, x.y), Elem<T>::pack(x.z, x.w));
                else reinterpret_cast<float4 *>(g.s.o + (long long)seg * g.sp.zg * D)[i] = x;
            }
        }
        p.t += cnt;
        if (p.t >= t1) break;
        next_row<D>(c, g.sp.blocks, p);
    }
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// (reference, sum of w) over a row's segments of one head (the whole warp calls it).
template <bool RELATIVE>
__device__ __forceinline__ float2 join_sums(const float2 *at, int zg, int count) {
    float2 x = make_float2(kLowest, 0.f);
#pragma unroll 2
    for (int i = threadIdx.x & 31; i < count; i += 32) x = join<RELATIVE>(x, __ldcg(at + (long long)i * zg));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = join<RELATIVE>(x, shuffle_xor(x, o));
    return x;
}

// Blocks [0, join_blocks): the output rows of several segments and those of
// sequences that are empty (zeros) or unusable (NaN), `warps_per` warps for each
// query head; the others: the scores, each block an equal run of the tiles
// numbered through (sequence, key head, tile).  Everything that the lengths alone
// decide is done before the wait for the kernel that this one depends on.
template <typename T, int D, int MODE, bool SCORES>
__global__ void __launch_bounds__(kJoinThreads, 4) paged_join(const __grid_constant__ Args g, int join_blocks, int warps_per) {
    constexpr int kPerLane = D / 32, kTile = tile_keys(D);
    constexpr bool kRelative = !is_reweight(MODE);
    const PagedCache &c = g.a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = g.sp.G;
    const int per_row = tiles_before<D>(c, c.B), total = per_row * g.sp.heads_rows, run = max(1, (total + g.sp.ctas - 1) / g.sp.ctas);
    if (!SCORES || (int)blockIdx.x < join_blocks) {
        __shared__ float part[kJoinWarps][D];
        const int sub = warp % warps_per, r = blockIdx.x * (kJoinWarps / warps_per) + warp / warps_per;
        const bool live = r < c.B * g.a.H;
        const int b = live ? r / g.a.H : 0, hq = live ? r % g.a.H : 0, h = hq / G, gq = hq % G;
        const int n = paged_len(c, b), nt = tiles_of<D>(n), hr = h * g.sp.blocks + gq / kHeads;
        Segments sg = {0, 0};
        if (live && n > 0) sg = segments_of(b * g.sp.heads_rows + hr, tiles_before<D>(c, b) * g.sp.heads_rows + hr * nt, nt, run);
        if (!dcheck(sg.first + sg.count <= segments_of_all(g), c.err, kDbgItem)) sg = {0, 0};
        const float2 *sums = g.s.sums + (long long)sg.first * g.sp.zg + gq % kHeads;
        const float *o = g.s.o + ((long long)sg.first * g.sp.zg + gq % kHeads) * D + lane * kPerLane;
        ptx::grid_dependency_wait();
        float acc[kPerLane];
#pragma unroll
        for (int e = 0; e < kPerLane; ++e) acc[e] = 0.f;
        if (sg.count > 1) {
            const float2 all = join_sums<kRelative>(sums, g.sp.zg, sg.count);
            const float inv = ptx::rcp(all.y);
#pragma unroll 4
            for (int i = sub; i < sg.count; i += warps_per) {
                const float f = kRelative ? inv * ptx::ex2(__ldcg(sums + (long long)i * g.sp.zg).x - all.x) : inv;
                const float *from = o + (long long)i * g.sp.zg * D;
                if constexpr (kPerLane == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(from));
                    acc[0] = fmaf(v.x, f, acc[0]);
                    acc[1] = fmaf(v.y, f, acc[1]);
                    acc[2] = fmaf(v.z, f, acc[2]);
                    acc[3] = fmaf(v.w, f, acc[3]);
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(from));
                    acc[0] = fmaf(v.x, f, acc[0]);
                    acc[1] = fmaf(v.y, f, acc[1]);
                }
            }
        }
        if (warps_per > 1) {
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) part[warp][lane * kPerLane + e] = acc[e];
            __syncthreads();
            if (sub) return;
#pragma unroll 1
            for (int w = 1; w < warps_per; ++w)
#pragma unroll
                for (int e = 0; e < kPerLane; ++e) acc[e] += part[warp + w][lane * kPerLane + e];
        }
        if (!live || sg.count == 1) return;   // written with its segment
        if (n == 0) {
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) acc[e] = c.lens[b] ? NAN : 0.f;
        }
        uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(g.a.out) + (long long)r * D + lane * kPerLane);
#pragma unroll
        for (int e = 0; e < kPerLane; e += 2) out[e / 2] = Elem<T>::pack(acc[e], acc[e + 1]);
        return;
    }
    if constexpr (SCORES) {
    // four slots per thread
    __shared__ float2 rowf[kMaxGroup];   // the sums' joint reference, 1 / sum of w
    constexpr int kThreads = kTile / 4, kStep = kJoinThreads / kThreads;
    const int keys = per_row * c.Hkv, blocks = gridDim.x - join_blocks, krun = (keys + blocks - 1) / blocks;
    const int t0 = (blockIdx.x - join_blocks) * krun, t1 = min(keys, t0 + krun);
    Place p = {};
    if (t0 < t1) p = locate<D>(c, 1, t0);
    p.t = t0;
    const bool vec = ((reinterpret_cast<uintptr_t>(g.a.scores) | reinterpret_cast<uintptr_t>(g.a.scores_out)) & 15) == 0;
    const int in = (threadIdx.x % kThreads) * 4;
    ptx::grid_dependency_wait();
#pragma unroll 1
    while (p.t < t1) {
        const int cnt = min(t1 - p.t, p.nt - p.tile);
        // number of the row's first tile among the stream's: the rows before it, each `blocks` times
        const int start = (p.t - p.tile - p.h * p.nt) * g.sp.blocks + p.h * g.sp.blocks * p.nt;
        const size_t base = ((size_t)p.b * c.Hkv + p.h) * c.capacity() + (size_t)p.tile * kTile + in;
        if (!dcheck(in_numbering<D>(g, p, cnt) && start + g.sp.blocks * p.nt <= c.B * g.sp.heads_rows * tiles_of<D>(c.capacity()), c.err, kDbgItem)) break;
        __syncthreads();
#pragma unroll 1
        for (int x = warp; x < G; x += kJoinWarps) {
            const Segments sg = segments_of(p.b * g.sp.heads_rows + p.h * g.sp.blocks + x / kHeads, start + x / kHeads * p.nt, p.nt, run);
            const float2 all = join_sums<kRelative>(g.s.sums + (long long)sg.first * g.sp.zg + x % kHeads, g.sp.zg, sg.count);
            if (lane == 0) rowf[x] = make_float2(all.x, ptx::rcp(all.y) * (MODE == kLssa ? ptx::ex2(-all.x) : 1.f));
        }
        __syncthreads();
#pragma unroll 1
        for (int i = threadIdx.x / kThreads; i < cnt; i += kStep) {
            const int have = p.n - (p.tile + i) * kTile - in;
            if (have <= 0) continue;
            const size_t at = base + (size_t)i * kTile;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f), add = s;
            if (vec && have >= 4) s = __ldcg(reinterpret_cast<const float4 *>(g.a.scores + at));
#pragma unroll 4
            for (int x = 0; x < G; ++x) {
                const long long tile = start + x / kHeads * p.nt + p.tile + i;
                float4 w = __ldcg(reinterpret_cast<const float4 *>(&g.s.z[(tile * g.sp.zg + x % kHeads) * kTile + in]));
                const float2 f = rowf[x];
                if (!is_reweight(MODE)) {
                    const float2 a = weights<MODE>(make_float2(w.x, w.y), f.x, 1.f), b = weights<MODE>(make_float2(w.z, w.w), f.x, 1.f);
                    w = make_float4(a.x, a.y, b.x, b.y);
                }
                add = make_float4(fmaf(w.x, f.y, add.x), fmaf(w.y, f.y, add.y), fmaf(w.z, f.y, add.z), fmaf(w.w, f.y, add.w));
            }
            if (vec && have >= 4) {
                *reinterpret_cast<float4 *>(g.a.scores_out + at) = make_float4(s.x + add.x, s.y + add.y, s.z + add.z, s.w + add.w);
            } else {
#pragma unroll 1
                for (int k = 0; k < min(have, 4); ++k)
                    g.a.scores_out[at + k] = g.a.scores[at + k] + (k == 0 ? add.x : k == 1 ? add.y : k == 2 ? add.z : add.w);
            }
        }
        p.t += cnt;
        if (p.t < t1) next_row<D>(c, 1, p);
    }
    }
}

inline cudaError_t launch_kernel(const void *fn, int grid, int block, size_t smem, bool dependent, void **args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

template <typename T, int D, int MODE, int PHASE>
cudaError_t launch_phase(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, bool dependent, cudaStream_t stream) {
    static PerDeviceOnce once;
    const void *fn = (const void *)paged_stream<T, D, MODE, PHASE>;
    constexpr int smem = Config<D, PHASE>::kSmem;
    const cudaError_t e = per_device_once(once, nullptr, [&](int &) { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    void *args[] = {(void *)&km, (void *)&vm, (void *)&g};
    return launch_kernel(fn, g.sp.ctas, kBlock, smem, dependent, args, stream);
}

template <typename T, int D, int MODE>
cudaError_t launch_mode(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t stream) {
    cudaError_t e;
    if constexpr (is_reweight(MODE)) {
        e = launch_phase<T, D, MODE, kScores>(km, vm, g, false, stream);
        if (e == cudaSuccess) e = launch_phase<T, D, MODE, kValues>(km, vm, g, true, stream);
    } else {
        e = launch_phase<T, D, MODE, kBoth>(km, vm, g, false, stream);
    }
    if (e != cudaSuccess) return e;
    // a block for each query head while there are few (their rows have many segments), else a warp
    const int rows = g.a.c.B * g.a.H;
    int warps_per = rows <= sms ? kJoinWarps : 1, join_blocks = (rows * warps_per + kJoinWarps - 1) / kJoinWarps;
    const int blocks = join_blocks + (g.a.scores ? (g.sp.ctas < 3 * sms ? g.sp.ctas : 3 * sms) : 0);
    void *args[] = {(void *)&g, (void *)&join_blocks, (void *)&warps_per};
    const void *fn = g.a.scores ? (const void *)paged_join<T, D, MODE, true> : (const void *)paged_join<T, D, MODE, false>;
    return launch_kernel(fn, blocks, kJoinThreads, 0, true, args, stream);
}

// One call per (type, d) and file, so that the instances compile in parallel.
#define LSSAR_PAGED_DECODE_INSTANCES(T, D, NAME)                                                                        \
    cudaError_t NAME##_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t st) {  \
        switch (g.a.mode) {                                                                                             \
            case kSoftmax: return launch_mode<T, D, kSoftmax>(km, vm, g, sms, st);                                      \
            case kLssa: return launch_mode<T, D, kLssa>(km, vm, g, sms, st);                                            \
            case kLssar: return launch_mode<T, D, kLssar>(km, vm, g, sms, st);                                          \
            case kSoftmaxRw: return launch_mode<T, D, kSoftmaxRw>(km, vm, g, sms, st);                                  \
            default: return launch_mode<T, D, kSigmoidRw>(km, vm, g, sms, st);                                          \
        }                                                                                                               \
    }

cudaError_t bf16_d64_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t st);
cudaError_t bf16_d128_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t st);
cudaError_t fp16_d64_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t st);
cudaError_t fp16_d128_launch(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t st);

}  // namespace paged
}  // namespace lssar
