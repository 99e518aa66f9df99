// Paged cache, attention of a chunk: the last counts[b] rows of the attention over the
// lens[b] cached tokens of each sequence, in every mode, grouped heads.
//
// Mathematics, for row i (tokens it attends to) and key j < i, in log2 units:
//   z = log2e / sqrt(d) q.k  (softmax modes)  or  log2e ln d ln i q.k / (|q| |k|);
//   phi(z) = 2^(z - m), log2(1 + 2^z) or 1 / (1 + 2^-z);  S1 = sum phi, m = max z;
//   w = phi, or re-weighted max(kappa (phi - theta), 0)^p, theta = O S1 / i,
//   kappa = 1 / (phi(m) - theta);  out = sum w v / sum w.
// Scores are products of the inputs' own bits, scaled in fp32 afterwards: 1/|k| of each cached
// key comes from a prologue that reads them once, |q| from the gathered rows.
//
// What bounds it: the score warps.  For 32 scores the statistics pass executes 7.1 warp instructions (4.9 of them
// arithmetic, one a special function), the values pass at p = 15 11.7 (7.4); the others are branches, waits, indices
// and loads.  Against that stand 4 d flops of tensor work a score and, at 256 rows per key, 4 d / 256 bytes.
// Measured (kernels alone): 2K rows on 14K tokens, 12 heads of 64, LSSAR p = 15: 103 + 181 us (issue slots
// 66 and 61 % busy, so that what is executed would fill 71 and 116 us; tensor pipe 20 and 23 %); 512 rows on 128K,
// 16/2 heads of 128: 270 + 500 us (69 and 57 %, tensor 43 and 46 %); four prompts of 4K, 16 heads of 128, LSSA: 350 us
// (47 %, tensor 38 %), softmax 308 us, where the dense forward, with its one MMA warp, products 128 keys wide and (LSSA)
// normalised copies of the rows, takes 242 and 229.
// The time depends on the scores: rows whose scores are all negative take the softplus evenly to its own value
// (kAccurate, and the statistics twice): the 2K rows above take the call 537 us instead of 303.
//
// Split.  A work item is a pair of 128-row tiles of the rows (token, head of the group) of one
// key head: floor(256 / G) tokens.  What an item costs, its K tiles of 128 keys and a share for its own beginning
// and end, is numbered through in units (sequence, pair, key head, tile); each CTA takes an equal run of them
// wherever items begin or end, as in the decode step, so that chunks and contexts of any mix load the SMs evenly.
// The part of an item in one run is a segment.  The numbering needs the lengths, which are on the device:
//   attend_prepare   plans it (one block), while the other blocks work out the norms;
//   attend<kStats>   re-weighting modes: scores -> (m, S1) of each segment's rows;
//   attend<kValues>  row constants from all of the item's segments, scores again,
//                    weights, sum of w v; writes the rows of whole items;
//   attend_join      adds the segments of the items that lie in several runs.
// Each is a programmatic dependent of the one before it.  Small calls are their latencies: 64 rows on 200 tokens
// take 27.5 us of device time (shortest runs of 5, 9, 12 or 16 units in place of 2: 30, 29, 41, 43; 28 where a CTA
// finds its first entry, and that entry's lengths, by further reads).
//
// Structure of attend (640 threads): warp 0 the TMA producer of K (a piece of a page at a time) and of
// key norms, warp 3 that of V (one producer for both: 397 us in place of 393 on the prompts, and 29.5 in place of
// 26.8 on pages of 24 rows); warps 1, 2 issue the tcgen05.mma of one tile each; four warpgroups of score
// warps, two per tile, each half of its columns: thread = row (TMEM lane).  They also gather the rows of q
// (any strides, any group) of the next segment during the last step of this one.  Warps whose 32 rows hold none of
// the item's skip the arithmetic.  An item of one tile of rows has them in both row slots, which take turns with its
// tiles of keys and add up at the end (16 ragged sequences, 32/8 heads of 128: 77 -> 69 us).
// TMEM (512 columns): kStats: S of tile w, two buffers each, at 256 w + 128 buffer.  kValues: S_w at
// 128 w; d = 64: P_w at 256 + 64 w, O_w at 384 + 64 w; d = 128: P_w over S_w, O_w at 256 + 128 w.
#pragma once

#include <cstddef>

#include "paged_decode.cuh"
#include "tc_kernel.cuh"

namespace lssar {
namespace attend {

using tc::max3;
using tc::min3;

enum Phase : int { kStats = 0, kValues = 1 };

constexpr int kTileRows = 128;
constexpr int kPairRows = 256;
constexpr int kKeys = 128;                    // keys per tile
constexpr int kThreads = 640;
constexpr int kScoreWarp0 = 4;
// Registers: the control warpgroup gives some back, the score warpgroups take them
// (128 x 64 + 512 x 104 = 640 x 96).
constexpr int kLaunchRegs = 96, kCtrlRegs = 64, kScoreRegs = 104;
static_assert(128 * kCtrlRegs + 512 * kScoreRegs <= kThreads * kLaunchRegs, "register split");
// Tiles whose key norms are in shared memory.  They come with the tile's keys, and the place of tile j's is used
// again for tile j + 16, which waits until both MMA warps have passed tile j + 8 (kStats, d = 64; the others have
// fewer stages).  A row slot that still reads the norms of j is in j's item, so that the queue of kItems holds the
// eight tiles after j in that item and three more at most; of n tiles of one of them the slot takes n or n / 2
// (rounded down), two or more of the eight in all; and the second product of scores after j's waits
// for s_free of j's, which follows the reading of its norms.
constexpr int kInfo = 16;
constexpr int kItems = 4;                     // depth of the queue of segments
// What a work item costs, in the units that its run is counted in: of each tile of keys, and beside them (these
// are numbered before its first tile).  An item of one tile of rows takes a tile of keys in half the time.  (Items
// of both kinds at 6, units: ragged 68.5 us, pages of 24 18.8 us; 4: 67.4, 21.2; 8: 71.8, 19.9; none at all: prompts
// 393 us in place of 360.)
__host__ __device__ constexpr int tile_cost(int rows) { return rows > 128 ? 2 : 1; }
constexpr int kItemCost = 6;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint32_t kNapProducer = 200;   // ns between its polls of a barrier
constexpr float kLowest = -3.0e38f;           // below every score, and finite
enum : unsigned { kErrItem = 61, kErrQ, kErrKvFull, kErrKvEmpty, kErrSFull, kErrSFree, kErrPFull, kErrPFree, kErrOFull, kErrOFree,
                  kErrHalves, kErrTileMax, kErrDrain, kErrJoint };

// One-pass modes: log2 of the largest weight of a row lies in kRoom + [0, kLag] (fp16, whose
// least step is 2^-24, needs the room; softplus up to 117 leaves less of it; softmax's raises, with 13 and a
// lag of 2, took 140 us instead of 132 on 512 rows on 32K, d = 128).
template <int MODE, bool HALF>
struct Range16 {
    static constexpr float kRoom = !HALF ? 0.f : MODE == kSoftmax ? 12.f : 8.f;
    static constexpr float kLag = !HALF ? 8.f : MODE == kSoftmax ? 3.875f : 6.f;
};
constexpr float kTopFp16 = 32768.f;           // re-weighting: the largest weight in fp16
constexpr float kNoLift = -118.f;             // LSSA: below every score

struct Header {
    int total, entries, run;                  // units of cost, entries, units per CTA
};

struct Scratch {
    Header *head;
    int4 *entries;        // {sequence, pair, cost of an item, number of the first item's first unit}
    int4 *first;          // [ctas][2]: the entry of each CTA's first unit; its number, new tokens, cached tokens
    float *knorm;         // [B, Hkv, cap128] 1 / |k|
    float2 *stats;        // [item + cta][rows]: m, S1 of a segment's rows
    float2 *sums;         // [2 cta + last][rows]: reference, sum of w
    float *o;             // [2 cta + last][rows][d]: sum of w v
};

// The exponent, itself and as 3^cubes * rest.
struct Power {
    int exact, cubes, rest;
};

struct Args {
    PagedAttend a;
    Scratch s;
    int G, tokens;        // H / Hkv, tokens per pair
    int ctas, rows;       // rows that a segment's scratch holds
    int cap128;           // capacity, a multiple of 128
    int piece_rows;       // rows of a page per copy
    float scale;          // log2e / sqrt(d), or +-log2e ln d
    int exact_weights;    // 1: LSSAR rows never take the one-exponential weights
    Power power;
    uint32_t idesc_s, idesc_s64, idesc_pv;     // scores of 128 keys, of 64; sum of w v
};

// A segment as the roles of a CTA see it.
struct Item {
    int b, h, t0, rows;   // first token, valid rows of the pair
    int base, len;        // slots before the chunk, cached tokens
    int nk, kt0, kt1;     // tiles of the item; those of this segment
    int step;             // 2: one tile of rows, whose keys both row slots share, every other tile
    int item, start;      // number of the item, of its first tile's first unit (its cost comes before)
    int first_bad;        // first slot of a page that is none
};

struct __align__(16) Shared {
    float knorm[kInfo][kKeys];
    float m[2][2][2][kTileRows], s[2][2][2][kTileRows];   // [meeting parity][tile][half][row]
    float qq[2][2][2][kTileRows];                         // sum of squares of the next row of q, likewise
    float tmax[2][2][2][kTileRows];                       // [step parity, or kTurns: 1 for references][tile][half][row]
    float other[2][kTileRows][2];                         // [join parity][row]: the second slot's sums
    uint64_t q_full[2];
    uint64_t s_full[2][2], s_free[2][2];                  // [tile][buffer], or (kSplit) [tile][half]
    uint64_t p_full[2], p_free[2], o_full[2], o_free[2], halves[2], joint;
    uint64_t tile_max[2][4], turn[2][2][4];               // [half][tile][quarter]
    uint64_t kv_full[8], kv_empty[8];
    uint64_t item_full[kItems], item_empty[kItems];
    Item items[kItems];
    unsigned absent[8];   // per stage of V: groups of 8 rows that no copy has filled
    uint32_t tmem;
    int abort_flag;
};

template <int D>
struct Cfg {
    static constexpr int kTile = kTileRows * D * 2;      // bytes of a tile of q, k or v
    static constexpr int kStages = D == 64 ? 8 : 4;
    static constexpr int kRing = 2 * kTile;              // behind the two tiles of q
    static constexpr int kShared = kRing + kStages * kTile;
    static constexpr int kSmem = kShared + (int)sizeof(Shared) + 1024;
};
static_assert(Cfg<64>::kSmem <= 232448 && Cfg<128>::kSmem <= 232448, "shared memory");

// Rows of the pair that starts at token t0, of a sequence with `count` new tokens.
__device__ __forceinline__ int rows_of_pair(const Args &g, int count, int t0) { return min(g.tokens, count - t0) * g.G; }

// Tiles of a pair that starts at token t0, of a sequence with `count` new tokens after `base`.
__host__ __device__ __forceinline__ int tiles_of_pair(int base, int count, int t0, int tokens) {
    const int last = t0 + tokens < count ? t0 + tokens : count;     // tokens up to the pair's end
    return (base + last + kKeys - 1) / kKeys;
}

// Sum of squares of 8 elements.
__device__ __forceinline__ float squares(uint4 x, bool half) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = half ? __half22float2(*reinterpret_cast<const __half2 *>(&u[i]))
                              : make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
        s = fmaf(f.x, f.x, fmaf(f.y, f.y, s));
    }
    return s;
}

// ---------------------------------------------------------------- prologue

constexpr int kPrepThreads = 256;

// Exclusive prefix over the block of two values; the totals in t0, t1.
__device__ __forceinline__ void block_prefix(long long &x, long long &y, long long &tx, long long &ty, long long (*part)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ax = __shfl_up_sync(0xffffffffu, ix, o), ay = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) {
            ix += ax;
            iy += ay;
        }
    }
    __syncthreads();
    if (lane == 31) {
        part[warp][0] = ix;
        part[warp][1] = iy;
    }
    __syncthreads();
    tx = ty = 0;
    x = ix - x;
    y = iy - y;
#pragma unroll
    for (int w = 0; w < kPrepThreads / 32; ++w) {
        if (w < warp) {
            x += part[w][0];
            y += part[w][1];
        }
        tx += part[w][0];
        ty += part[w][1];
    }
}

// The plan (one block): entries in the order of (sequence, pair), and each CTA's first one.
static __device__ __noinline__ void make_plan(const Args &g) {
    __shared__ long long part[kPrepThreads / 32][2];
    __shared__ int bad[kPrepThreads];
    const PagedAttend &a = g.a;
    const PagedCache &c = a.c;
    long long entries = 0, tiles = 0;
#pragma unroll 1
    for (int base = 0; base < c.B; base += kPrepThreads) {
        const int b = base + threadIdx.x;
        int len = 0, cnt = 0;
        bool ok = true;
        if (b < c.B) {
            len = c.lens[b];
            cnt = a.counts ? a.counts[b] : a.n;
            ok = len >= 0 && len <= c.capacity() && cnt >= 0 && cnt <= a.n && cnt <= len;
            if (!ok) {
                atomicCAS(c.err, 0u, (unsigned)kErrPagedLength);
                cnt = 0;
            }
        }
        const int pairs = (cnt + g.tokens - 1) / g.tokens;
        long long mine = 0;
#pragma unroll 1
        for (int m = 0; m < pairs; ++m) {
            const int rows = rows_of_pair(g, cnt, m * g.tokens);
            mine += kItemCost + tile_cost(rows) * tiles_of_pair(len - cnt, cnt, m * g.tokens, g.tokens);
        }
        long long e = pairs, t = mine * c.Hkv, te, tt;
        block_prefix(e, t, te, tt, part);
        e += entries;
        t += tiles;
#pragma unroll 1
        for (int m = 0; m < pairs; ++m) {
            const int rows = rows_of_pair(g, cnt, m * g.tokens);
            const int cost = kItemCost + tile_cost(rows) * tiles_of_pair(len - cnt, cnt, m * g.tokens, g.tokens);
            g.s.entries[e++] = make_int4(b, m, cost, (int)t);
            t += (long long)cost * c.Hkv;
        }
        entries += te;
        tiles += tt;
        // rows of a sequence that must not be used
        bad[threadIdx.x] = !ok;
        if (__syncthreads_or(!ok)) {
#pragma unroll 1
            for (int i = 0; i < min(kPrepThreads, c.B - base); ++i) {
                if (!bad[i]) continue;
                uint4 *row = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (size_t)(base + i) * a.H * a.n * c.d);
                const size_t pieces = (size_t)a.H * a.n * c.d / 8;
                for (size_t x = threadIdx.x; x < pieces; x += kPrepThreads) row[x] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            }
        }
    }
    __syncthreads();
    const int run = max(2, (int)((tiles + g.ctas - 1) / g.ctas));      // (2: a tile's last unit lies in every run)
    if (threadIdx.x == 0) *g.s.head = Header{(int)tiles, (int)entries, run};
    for (int cta = threadIdx.x; cta < g.ctas; cta += kPrepThreads) {
        const long long t = (long long)cta * run;
        if (t >= tiles) break;
        int lo = 0, hi = (int)entries - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (g.s.entries[mid].w <= t) lo = mid;
            else hi = mid - 1;
        }
        const int4 en = g.s.entries[lo];
        g.s.first[2 * cta] = en;
        g.s.first[2 * cta + 1] = make_int4(lo, a.counts ? a.counts[en.x] : a.n, c.lens[en.x], 0);
    }
}

// Block 0 plans; the others, in the normalised modes, take runs of key rows: 1 / |k|.  2d bytes of each are
// read once, by d / 8 lanes a row.
template <int D>
__global__ void __launch_bounds__(kPrepThreads) attend_prepare(const __grid_constant__ Args g, int norms) {
    ptx::launch_dependents();
    if (blockIdx.x == 0) {
        make_plan(g);
        return;
    }
    if (!norms) return;
    const PagedAttend &a = g.a;
    const PagedCache &c = a.c;
    constexpr int kLanes = D / 8, kRows = kPrepThreads / kLanes, kTile = paged::tile_keys(D);
    const int part = threadIdx.x % kLanes, in = threadIdx.x / kLanes, blocks = gridDim.x - 1, blk = blockIdx.x - 1;
    // keys
    const int tiles = paged::tiles_before<D>(c, c.B) * c.Hkv, run = (tiles + blocks - 1) / blocks;
    const int t0 = blk * run, t1 = min(tiles, t0 + run);
    if (t0 < t1) {
        paged::Place p = paged::locate<D>(c, 1, t0);
#pragma unroll 1
        for (int t = t0; t < t1; ++t) {
            uint4 x[kTile / kRows];
#pragma unroll
            for (int e = 0; e < kTile / kRows; ++e) {
                const int slot = p.tile * kTile + e * kRows + in, i = slot / c.page_size;
                const int pg = slot < p.n ? c.table[(size_t)p.b * c.max_pages + i] : -1;
                x[e] = make_uint4(0, 0, 0, 0);
                if ((unsigned)pg < (unsigned)c.n_pages)
                    x[e] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(c.k) + pg * c.page_stride +
                                                            ((size_t)p.h * c.page_size + slot - i * c.page_size) * D + part * 8);
            }
#pragma unroll
            for (int e = 0; e < kTile / kRows; ++e) {
                float s = squares(x[e], c.half);
#pragma unroll
                for (int o = kLanes / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                const int slot = p.tile * kTile + e * kRows + in;
                if (part == 0 && slot < p.n) g.s.knorm[((size_t)p.b * c.Hkv + p.h) * g.cap128 + slot] = 1.f / fmaxf(sqrtf(s), 1e-12f);
            }
            if (++p.tile == p.nt && t + 1 < t1) paged::next_row<D>(c, 1, p);
        }
    }
}

// ---------------------------------------------------------------- scores

// A row's state; the score scale is negative in the sigmoid mode, whose registers hold -z.
struct Row {
    float a;
    float x;        // softmax: reference of the exponent less the room; LSSA: 2^(room - reference); else lift
    float ref;      // one pass: the reference
    float kappa, beta, theta, ck;
};

// Four key norms of a tile.  Volatile: between the waits and arrivals around it.
__device__ __forceinline__ float4 load_norms(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float2 pair_at(const uint32_t *r, int j) { return make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])); }

// Products of N columns -> z; `knorm`: the norms of the first.
template <bool NORM, int N>
__device__ __forceinline__ void to_z(uint32_t (&r)[N], uint32_t knorm, float a) {
    if constexpr (!NORM) {
        // Scores of any size, re-weighted softmax: each is rounded, as the row's maximum was, before the maximum is
        // taken from it.  (One by one: the compiler puts products of pairs and their sums into FMAs.)
#pragma unroll
        for (int j = 0; j < N; ++j) r[j] = __float_as_uint(__fmul_rn(__uint_as_float(r[j]), a));
        return;
    }
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        const float4 k = load_norms(knorm + j * 4);
        const float2 z0 = __fmul2_rn(pair_at(r, j), __fmul2_rn(make_float2(k.x, k.y), make_float2(a, a)));
        const float2 z1 = __fmul2_rn(pair_at(r, j + 2), __fmul2_rn(make_float2(k.z, k.w), make_float2(a, a)));
        r[j] = __float_as_uint(z0.x);
        r[j + 1] = __float_as_uint(z0.y);
        r[j + 2] = __float_as_uint(z1.x);
        r[j + 3] = __float_as_uint(z1.y);
    }
}

// Columns past `last` (relative to this chunk) get no weight.  (The empty instruction keeps the caller's
// branch: as selects it cost two instructions for each score of every tile.)
__device__ __forceinline__ void mask(uint32_t (&r)[32], int last, float masked) {
    asm volatile("");
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j > last) r[j] = __float_as_uint(masked);
}

__device__ __forceinline__ float max_of(const uint32_t (&r)[32], float m) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) m = max3(m, __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
    return m;
}

// sum phi of a chunk, LSSAR: sum max(z, 0) in acc and prod (1 + 2^-|z|) in prod, one special
// function a score (as the dense forward); or, ACCURATE, where all of a row's scores of the tile are
// negative, and the product would lose them, softplus itself.
template <bool ACCURATE>
__device__ __forceinline__ void softplus_sum(const uint32_t (&r)[32], float2 &acc, float2 &prod) {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 z = pair_at(r, j);
        if constexpr (ACCURATE) {
            acc = __fadd2_rn(acc, softplus2(z));
        } else {
            const float2 u = make_float2(ptx::ex2(-fabsf(z.x)), ptx::ex2(-fabsf(z.y)));
            prod = __ffma2_rn(prod, u, prod);
            acc = __fadd2_rn(acc, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
        }
    }
}

// x[i]^p, 16 values at once.  P = 3 and 15, the exponents of the method's own results, unrolled; others by loops
// over 3^cubes * rest, the same for all threads (their branches cost two instructions for each score).
template <int P>
__device__ __forceinline__ void powers16(float2 (&x)[8], Power pw) {
    if constexpr (P == 3 || P == 15) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 c = __fmul2_rn(x[i], __fmul2_rn(x[i], x[i]));
            if constexpr (P == 3) {
                x[i] = c;
            } else {
                const float2 d = __fmul2_rn(c, c);
                x[i] = __fmul2_rn(c, __fmul2_rn(d, d));
            }
        }
        return;
    }
    float2 s[8];
#pragma unroll 1
    for (int c = pw.cubes; c > 0; --c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], __fmul2_rn(x[i], x[i]));
    }
    int p = pw.rest;
#pragma unroll 1
    for (; !(p & 1); p >>= 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], x[i]);
    }
    if (p == 1) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = __fmul2_rn(x[i], x[i]);
#pragma unroll 1
    for (p >>= 1;;) {
        if (p & 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], s[i]);
        }
        if ((p >>= 1) == 0) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = __fmul2_rn(s[i], s[i]);
    }
}

// How a warp evaluates its weights (a warp-uniform choice).
enum Form : int {
    kMixed = 0,      // softplus by logarithms and a polynomial in turn, to about 2^-19 (1 + its value)
    kOneExp = 1,     // LSSAR rows that meet the bound of fast_weights.cuh (none with LSSAR_EXACT_WEIGHTS=1)
    kAccurate = 2    // to 2^-18 of its value and evenly: rows whose scores are all negative, or nearly equal;
                     // softmax: rows whose scores pass 2^16
};

// Of every 16 pairs, those whose softplus takes the polynomial: the rest of the work leaves the FMA pipe
// more room in LSSA.  (2K on 14K, 12 heads of 64, LSSA: 2 183 us, 5 173, 6 172, 8 167, 11 182; LSSAR p = 3: 2 and 4 194, 5
// to 11 201 to 204.)
template <int MODE>
constexpr int kPolyPairs = MODE == kLssa ? 8 : 4;

// Weights of 16 scores (r[0..15]), summed into acc and packed into 8 words.  `pair0`: number of the
// first pair in its chunk of 32.
// They are rounded to the type of the values, half a step (2^-8 of each in bf16, 2^-11 in fp16): a tensor product takes both
// operands in one type, and one more of what the rounding leaves would double the values' share of the tensor pipe.  The sum
// takes them in fp32, as they were: the roundings, of either sign, average over the row.  Error of the output against
// float64, in the norm, with fp32 weights and here: LSSA prompts 0.0016 and 0.0023, 64 rows on 200 0.0017 and
// 0.0018, the other chunks of bf16 (0.0016 and 0.0017) and of fp16 (0.00021) the same, as the output's own rounding is.
template <int MODE, bool HALF, int FORM, int P>
__device__ __forceinline__ void weights16(const uint32_t *r, int pair0, const Row &row, Power p, float2 &acc, uint32_t *pk) {
    const auto both = [](float x) { return make_float2(x, x); };
    float2 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 z = pair_at(r, 2 * i);
        if constexpr (MODE == kSoftmax || MODE == kSoftmaxRw) {
            // (softmax: z holds the product.  Beyond 2^16 its own rounding would pass the room: scaled first)
            const float2 e = MODE == kSoftmaxRw ? __fadd2_rn(z, both(-row.x))
                             : FORM == kMixed   ? __ffma2_rn(z, both(row.a), both(-row.x))
                                                : make_float2(__fmul_rn(z.x, row.a) - row.x, __fmul_rn(z.y, row.a) - row.x);
            w[i] = make_float2(ptx::ex2(e.x), ptx::ex2(e.y));
        } else if constexpr (MODE == kSigmoidRw) {   // z holds -z
            const float2 v = __fadd2_rn(make_float2(ptx::ex2(z.x), ptx::ex2(z.y)), both(1.f));
            w[i] = make_float2(ptx::rcp(v.x), ptx::rcp(v.y));
        } else if constexpr (FORM == kAccurate) {
            w[i] = softplus2(z);
        } else if constexpr (FORM == kOneExp) {
            const float2 u = make_float2(ptx::ex2(-fabsf(z.x)), ptx::ex2(-fabsf(z.y)));
            w[i] = ptx::fma_sat2(u, both(row.ck), __ffma2_rn(z, both(row.kappa), both(row.beta)));
        } else {
            w[i] = poly_pair(pair0 + i, kPolyPairs<MODE>) ? sp2x2_poly(z) : tc::sp2x2_direct(z);
        }
        if constexpr (is_reweight(MODE) && FORM != kOneExp) {
            // the difference before its scale where it is small against its terms (kAccurate)
            if constexpr (FORM == kAccurate) {
                const float2 y = MODE == kSoftmaxRw ? __fadd2_rn(w[i], both(-row.theta)) : __ffma2_rn(w[i], both(row.x), both(-row.theta));
                w[i] = ptx::fma_sat2(y, both(row.kappa), both(0.f));
            } else {
                w[i] = ptx::fma_sat2(w[i], both(row.kappa), both(row.beta));
            }
        } else if constexpr (MODE == kLssa && (FORM == kAccurate || HALF)) {
            w[i] = __fmul2_rn(w[i], both(row.x));
        }
    }
    if constexpr (is_reweight(MODE)) {
        powers16<P>(w, p);
        if constexpr (HALF) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __fmul2_rn(w[i], both(kTopFp16));
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        acc = __fadd2_rn(acc, w[i]);
        pk[i] = HALF ? ptx::pack_f16x2(w[i].x, w[i].y) : ptx::pack_bf16x2(w[i].x, w[i].y);
    }
}

// Calls f with the form, and the exponent that is unrolled or 0, as a type.  (Loops over a tile's scores inside f: with the
// choice made anew for each 32 scores, after their products had taken the norms in a block of its own, 512 rows on
// 128K took 591 us instead of 505.)
template <int FORM, int P>
struct Weights {
    static constexpr int kForm = FORM, kP = P;
};
template <int MODE, class F>
__device__ __forceinline__ bool with_form(int form, int p, F f) {
    if (form == kAccurate) return f(Weights<kAccurate, 0>());
    if (!is_reweight(MODE)) return f(Weights<kMixed, 0>());
    if (MODE == kLssar && form == kOneExp) return p == 15 ? f(Weights<kOneExp, 15>()) : f(Weights<kOneExp, 0>());
    if (p == 15) return f(Weights<kMixed, 15>());
    if (p == 3) return f(Weights<kMixed, 3>());
    return f(Weights<kMixed, 0>());
}

// Constants of a re-weighted row from its maximum and normaliser sum; returns the form that it
// needs.  A row is uniform where the largest difference is within 1e-5 of the maximum, as in the
// decode step.  Its weights: phi 2^126 clamped to 1, which is 1 for every score that is not masked.
template <int MODE>
__device__ __forceinline__ int row_constants(Row &row, float m, float s1, int n, int p, bool exact_weights) {
    const bool raw = MODE == kSoftmaxRw;
    const float lift = raw ? 1.f : ptx::ex2(-fminf(m, 0.f));
    const float theta = n <= 3 ? 0.f : s1 * lift / (float)n;
    const float top = raw ? 1.f : MODE == kSigmoidRw ? sigmoid2(m) * lift : softplus2(make_float2(m, m)).x * lift;
    const float den = top - theta;
    row.x = raw ? m : lift;
    row.theta = theta;
    if (!(den > 1e-5f * top)) {
        row.theta = 0.f;
        row.kappa = tc::kUniformSlope;
        return isnan(s1) ? (row.kappa = NAN, kAccurate) : kAccurate;
    }
    row.kappa = ptx::rcp(den);
    row.beta = -theta * row.kappa;
    // the mixed form is off by 2^-19 (1 + phi): 2^-12 of the largest difference where that is 2^-7 of
    // the maximum or more, and the maximum is at least softplus(0)
    if (den < 0.0078125f * top || (!raw && m < 0.f)) return kAccurate;
    if constexpr (MODE == kLssar) {
        row.ck = 2.f * kHalfInvLn2 * row.kappa;
        if (!exact_weights && fast_weights_ok(theta, row.kappa, (float)n, p)) return kOneExp;
    }
    return kMixed;
}

// The shared block's members by 32-bit address (one register, constant offsets).
#define LSSAR_AT(member) (shared + (uint32_t)offsetof(Shared, member))

// A bounded wait that sleeps `nap` ns between polls: warps that poll without a pause took a third of the
// issue slots from the score warps.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint32_t shared, unsigned *err, unsigned code, uint32_t nap, bool honour_abort = true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
#pragma unroll 1
    for (uint32_t spin = 1;; ++spin) {
        if (nap) __nanosleep(nap);
        if (ptx::mbar_try_wait_sleep(bar, parity, 1000000)) return true;
        if ((spin & 63u) != 0) continue;
        if (honour_abort && ptx::ld_shared_s32(LSSAR_AT(abort_flag))) return false;
        if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicCAS(err, 0u, code);
            ptx::st_shared_s32(LSSAR_AT(abort_flag), 1);
            return false;
        }
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Row r of the tile of keys or values at `tile`: zeros.
template <int D>
__device__ __forceinline__ void clear_row(uint32_t tile, int r) {
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + (r >> 3) * (16 * D) + (x >> 3) * 1024 + (r & 7) * 128 + (x & 7) * 16), "r"(0) : "memory");
}

// A ring of `N` barriers: slot and parity of use number `i`.
template <int N>
struct Ring {
    uint32_t i = 0;
    __device__ __forceinline__ uint32_t slot() const { return i % N; }
    __device__ __forceinline__ uint32_t parity() const { return (i / N) & 1; }
    __device__ __forceinline__ bool reused() const { return i >= N; }
};

// The rows of q of the segment at shared address `it` for tile slot w: this thread's half of row `in`.
template <int D>
__device__ __noinline__ bool gather_rows(const Args &g, uint32_t it, uint32_t sq, int w, int half, int in) {
    const PagedAttend &a = g.a;
    auto next = [&](size_t offset) { return ptx::ld_shared_s32(it + (uint32_t)offset); };
    const int rows = next(offsetof(Item, rows)), kt0 = next(offsetof(Item, kt0)), shared_rows = next(offsetof(Item, step)) - 1;
    if (kt0 < 0 || kt0 + shared_rows * w >= next(offsetof(Item, kt1))) return false;
    const int v = min((shared_rows ? 0 : w * kTileRows) + in, rows - 1), tok = v / g.G, head = next(offsetof(Item, h)) * g.G + v - tok * g.G;
    const uint16_t *src = static_cast<const uint16_t *>(a.q) + next(offsetof(Item, b)) * a.qs[0] + head * a.qs[1] +
                          (next(offsetof(Item, t0)) + tok) * a.qs[2] + half * (D / 2);
    const uint32_t dst = sq + w * Cfg<D>::kTile + (D == 128 ? half * (kTileRows * 128) : 0) + in * 128;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
        const int piece = D == 128 ? x : half * 4 + x;
        cp_async16(dst + ((piece ^ (in & 7)) << 4), src + x * 8);
    }
    return true;
}

template <int D, int MODE, bool HALF, int PHASE>
__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, const __grid_constant__ Args g) {
    using C = Cfg<D>;
    constexpr int TB = C::kTile, kGroup = 16 * D;
    constexpr int NR = PHASE == kStats ? C::kStages : C::kStages / 2;       // stages of keys, and (kValues) of values
    constexpr bool kNorm = uses_normalised_qk(MODE);
    constexpr bool kOnePass = MODE == kSoftmax || MODE == kLssa;
    constexpr bool kSepP = D == 64;
    constexpr int kSBufs = PHASE == kStats ? 2 : 1;
    // kValues, d = 128: P lies over S, so that a product of scores waits for the weights of the one before.
    // The two halves of a tile's keys are then products of their own, and their warpgroups take turns (512 rows
    // on 128K, LSSAR: 737 -> 572 us).
    // Softmax: a half takes the reference of the turn before its own, which is the other half's, and raises it where
    // its own maximum asks for that: O is rescaled, all of its columns, between the two turns' products.  Only the first
    // tile's maxima meet (512 rows on 32K, 16/2 heads: 159 -> 134 us in bf16, 156 -> 132 in fp16; four prompts of 4K,
    // 16 heads: 345 -> 308; 16 ragged sequences, segments of 7 tiles: 71.7 -> 74.6; with the maxima of every tile
    // meeting, as products of their own, 84 in place of 77).
    constexpr bool kSplit = PHASE == kValues && !kSepP;
    constexpr bool kTurns = kSplit && MODE == kSoftmax;
    constexpr int kPCol = 256, kOCol = kSepP ? 384 : 256;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sq = ptx::smem_u32(smem), ring = sq + C::kRing;
    Shared *sh = reinterpret_cast<Shared *>(smem + C::kShared);
    const uint32_t shared = sq + C::kShared;
    const PagedAttend &a = g.a;
    const PagedCache &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned *err = c.err;

    if (threadIdx.x == 0) {
        auto init = [](uint64_t *b, uint32_t count) { ptx::mbar_init(ptx::smem_u32(b), count); };
        for (int i = 0; i < 2; ++i) {
            init(&sh->q_full[i], 256);
            for (int j = 0; j < 2; ++j) {
                init(&sh->s_full[i][j], 1);
                init(&sh->s_free[i][j], kSplit ? 128 : 256);
            }
            init(&sh->p_full[i], 256);
            init(&sh->p_free[i], 1);
            init(&sh->o_full[i], 1);
            init(&sh->o_free[i], 256);
            init(&sh->halves[i], 256);
            for (int j = 0; j < 4; ++j) {
                init(&sh->tile_max[i][j], 64);
                for (int h = 0; h < 2; ++h) init(&sh->turn[h][i][j], 32);
            }
        }
        init(&sh->joint, PHASE == kStats ? 256 : 512);
        for (int i = 0; i < 8; ++i) {
            init(&sh->kv_full[i], 1);
            init(&sh->kv_empty[i], 2);
        }
        for (int i = 0; i < kItems; ++i) {
            init(&sh->item_full[i], 1);
            init(&sh->item_empty[i], (PHASE == kValues ? 3 : 2) + 16);
        }
        sh->abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 1) {
        ptx::tmem_alloc(LSSAR_AT(tmem), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sh->tmem;
    // The plan, the norms and (kValues) the statistics are there from here on.  (What is launched next
    // may read the plan at once, and waits for the rest.)
    ptx::grid_dependency_wait();
    ptx::launch_dependents();

    const uint32_t nap = warp == 0 || warp == 3 ? kNapProducer : 0u;
    auto wait_all = [&](uint32_t bar, uint32_t parity, unsigned code) -> bool {
        return __all_sync(0xffffffffu, wait_bar(bar, parity, shared, err, code, nap));
    };
    // The next segment, or one with kt0 < 0 at the end; the slot is released by release_item.
    Ring<kItems> items;
    auto next_item = [&](Item &it) -> bool {
        if (!wait_all(LSSAR_AT(item_full) + 8 * items.slot(), items.parity(), kErrItem)) return false;
        it = sh->items[items.slot()];
        return it.kt0 >= 0;
    };
    auto release_item = [&] {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(LSSAR_AT(item_empty) + 8 * items.slot());
        ++items.i;
    };

    if (warp < kScoreWarp0) {
        if constexpr (PHASE == kValues) ptx::setmaxnreg_dec<kCtrlRegs>();
        if (warp == 0 || warp == 3) {
            // ------------------------------------------------------------ producers: keys (and the segments), values
            const bool keys = warp == 0;
            const CUtensorMap *map = keys ? &km : &vm;
            const int piece_rows = g.piece_rows, ps = c.page_size;
            const uint32_t first_stage = keys ? 0 : NR;
            Ring<NR> kv;
            bool ok = true;
            int pg = -1, row = 0;          // of this lane's piece of the tile looked up: page (-1 past the end, -2 no page), row
            Item it = {};
            if (ptx::elect_one()) ptx::prefetch_tensormap(map);
            auto look_up = [&](int kt) {
                const int s0 = kt * kKeys + lane * piece_rows, i = s0 / ps;
                pg = -1;
                if (lane * piece_rows >= kKeys || s0 >= it.len) return;
                row = it.h * ps + s0 - i * ps;
                pg = paged_page(c, it.b, i);
                if (pg < 0) pg = -2;
            };
            // the tiles of the segment, whose queue entry is `slot`
            auto load_tiles = [&](uint32_t slot) {
                look_up(it.kt0);
#pragma unroll 1
                for (int k = it.kt0; ok && k < it.kt1; ++k) {
                    const int page = pg, y = row;
                    if (k + 1 < it.kt1) look_up(k + 1);          // (arrives while this one waits for its stage)
                    const uint32_t s = first_stage + kv.slot(), full = LSSAR_AT(kv_full) + 8 * s;
                    if (kv.reused() && !(ok = wait_all(LSSAR_AT(kv_empty) + 8 * s, kv.parity() ^ 1, kErrKvEmpty))) break;
                    const unsigned there = __ballot_sync(0xffffffffu, page >= 0), bad = __ballot_sync(0xffffffffu, page == -2);
                    if (keys && bad) {
                        // keys of pages that are none: zeros, as rows that do attend to them have a say in the form of
                        // their warp's weights
                        for (int r = lane; r < kKeys; r += 32)
                            if (bad >> (r / piece_rows) & 1) clear_row<D>(ring + s * TB, r);
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) {
                        const int groups = piece_rows / 8;
                        unsigned absent = 0xffffu;
                        for (int i = 0; i * piece_rows < kKeys; ++i)
                            if (there >> i & 1) absent &= ~(((1u << groups) - 1) << (i * groups));
                        sh->absent[s] = absent;
                        if (keys && bad) {                        // the first slot of a page that is none
                            volatile int *first = &sh->items[slot].first_bad;
                            *first = min(*first, k * kKeys + (__ffs(bad) - 1) * piece_rows);
                        }
                        const bool norms = kNorm && keys;
                        ptx::mbar_arrive_expect_tx(full, (uint32_t)__popc(there) * piece_rows * D * 2 + (norms ? kKeys * 4 : 0));
                        const long long at = ((long long)it.b * c.Hkv + it.h) * g.cap128 + (long long)k * kKeys;
                        if (norms && dcheck((k + 1) * kKeys <= g.cap128 && it.b < c.B, err, kDbgBulk))
                            ptx::bulk_load(LSSAR_AT(knorm) + kv.i % kInfo * (kKeys * 4), g.s.knorm + at, kKeys * 4, full);
                    }
                    __syncwarp();
                    if (page >= 0 && dcheck(y >= 0 && y + piece_rows <= c.Hkv * ps && page < c.n_pages, err, kDbgTma))
                        ptx::tma_load_5d(ring + s * TB + lane * piece_rows * D * 2, map, full, 0, 0, 0, y >> 3, page);
                    ++kv.i;
                }
            };
            if (keys) {
                const Header head = *g.s.head;
                int4 en = g.s.first[2 * blockIdx.x], seq = g.s.first[2 * blockIdx.x + 1];      // (of a run without units: unused)
                const int t1 = min((long long)head.total, (long long)(blockIdx.x + 1) * head.run);
                long long t = (long long)blockIdx.x * head.run;
                int e = seq.x, h = 0, at = 0;       // the item, and the unit of it
                if (t < t1) {
                    h = (int)(t - en.w) / en.z;
                    at = (int)(t - en.w) - h * en.z;
                }
                while (ok) {
                    const uint32_t slot = items.slot();
                    if (items.reused() && !wait_all(LSSAR_AT(item_empty) + 8 * slot, items.parity() ^ 1, kErrItem)) break;
                    // the tiles of the item whose last unit lies in the run
                    it.kt0 = -1;
                    if (t < t1) {
                        const int cnt = seq.y;
                        it.b = en.x;
                        it.h = h;
                        it.t0 = en.y * g.tokens;
                        it.rows = rows_of_pair(g, cnt, it.t0);
                        it.len = seq.z;
                        it.base = it.len - cnt;
                        const int cost = kItemCost, each = tile_cost(it.rows), end = (int)min((long long)en.z, at + t1 - t);
                        it.nk = (en.z - cost) / each;
                        it.kt0 = max(at - cost, 0) / each;
                        it.kt1 = max(end - cost, 0) / each;
                        it.item = e * c.Hkv + h;
                        it.start = en.w + h * en.z + cost;
                        t += end - at;
                        at = 0;
                        it.step = it.rows > kTileRows ? 1 : 2;
                        it.first_bad = 0x7fffffff;
                        if (!dcheck(e < head.entries && h < c.Hkv && it.kt1 >= it.kt0 && it.rows > 0 && it.rows <= g.rows, err, kDbgItem)) it.kt0 = -1;
                        if (t < t1 && ++h == c.Hkv) {
                            h = 0;
                            en = g.s.entries[++e];
                            seq.y = a.counts ? a.counts[en.x] : a.n;
                            seq.z = c.lens[en.x];
                        }
                        if (it.kt0 >= 0 && it.kt0 == it.kt1) continue;      // none (part of the item's cost, of a tile's)
                    }
                    if (lane == 0) {
                        sh->items[slot] = it;
                        ptx::mbar_arrive(LSSAR_AT(item_full) + 8 * slot);
                    }
                    __syncwarp();
                    ++items.i;
                    if (it.kt0 < 0) break;
                    load_tiles(slot);
                }
            } else if constexpr (PHASE == kValues) {
                while (ok && next_item(it)) {
                    release_item();
                    load_tiles(0);
                }
            }
            // no copy may be in flight when the CTA ends
            for (uint32_t i = kv.i > NR ? kv.i - NR : 0; i < kv.i; ++i)
                wait_bar(LSSAR_AT(kv_full) + 8 * (first_stage + i % NR), (i / NR) & 1, shared, err, kErrDrain, nap, false);
            __syncwarp();
        } else {
            // ------------------------------------------------------------ MMA of tile w
            const int w = warp - 1;
            Ring<NR> keys, values;
            Ring<kSBufs> sb;               // S of this tile
            uint32_t pv = 0, qs = 0, segs = 0;     // P.V products issued; q tiles taken, segments ended, of this tile
            bool ok = true;
            auto commit = [&](uint32_t bar) {
                if (ptx::elect_one()) ptx::mma_commit(bar);
                __syncwarp();
            };
            // the stage of the next tile of keys, or of values
            auto acquire = [&](Ring<NR> &tiles, uint32_t first, uint32_t &stage) -> bool {
                stage = first + tiles.slot();
                if (!wait_all(LSSAR_AT(kv_full) + 8 * stage, tiles.parity(), kErrKvFull)) return false;
                ++tiles.i;
                ptx::tc_fence_after();
                return true;
            };
            const uint64_t dq0 = ptx::smem_desc_sw128(sq, tc::kKmajorLbo, tc::kKmajorSbo);
            // keys and values: groups of 8 rows, kGroup bytes apart, the 64-column blocks of a group 1024 bytes
            const uint64_t dk0 = ptx::smem_desc_sw128(ring, tc::kKmajorLbo, kGroup);
            const uint64_t dv0 = ptx::smem_desc_sw128(ring, 1024, kGroup);
            // S = q k^T of the K tile in kslot (its buffer is free once the score warps have read it)
            auto issue_s = [&](uint32_t kslot) -> bool {
                const uint32_t buf = sb.slot();
                if (sb.reused() && !wait_all((LSSAR_AT(s_free) + 16 * (w) + 8 * (buf)), sb.parity() ^ 1, kErrSFree)) return false;
                ptx::tc_fence_after();
                const uint64_t dq = dq0 + (uint64_t)((w * TB) >> 4), dk = dk0 + (uint64_t)((kslot * TB) >> 4);
                const uint32_t full = (LSSAR_AT(s_full) + 16 * (w) + 8 * (buf));
                const uint32_t col = tmem + (PHASE == kStats ? w * 256 + buf * kKeys : w * kKeys);
                dcheck(tmem_in_range(col, tmem, kKeys, 512), err, kDbgTmem);
                if (ptx::elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t q_off = ((k / 4) * 16384 + (k % 4) * 32) >> 4, k_off = ((k / 4) * 1024 + (k % 4) * 32) >> 4;
                        ptx::mma_ss(col, dq + q_off, dk + k_off, g.idesc_s, k > 0);
                    }
                    ptx::mma_commit(full);
                }
                __syncwarp();
                ++sb.i;
                return true;
            };
            // keys [from, from + 16 n) of the tile
            auto issue_pv = [&](uint32_t vslot, int from, int n, bool accumulate) {
                const uint64_t dv = dv0 + (uint64_t)((vslot * TB + from / 8 * kGroup) >> 4);
                const uint32_t words = kSepP ? tmem + kPCol + 64 * w + from / 2 : tmem + w * kKeys + from;
                if (ptx::elect_one()) {
#pragma unroll
                    for (int k = 0; k < n; ++k)
                        ptx::mma_ts(tmem + kOCol + w * D, words + 8 * k, dv + (uint64_t)((k * 2 * kGroup) >> 4), g.idesc_pv, (accumulate || k > 0) ? 1u : 0u);
                }
                __syncwarp();
            };
            // kSplit: scores of 64 keys
            auto issue_half = [&](uint32_t kslot, int h) {
                const uint64_t dq = dq0 + (uint64_t)((w * TB) >> 4), dk = dk0 + (uint64_t)((kslot * TB + h * 8 * kGroup) >> 4);
                const uint32_t full = LSSAR_AT(s_full) + 16 * w + 8 * h, col = tmem + w * kKeys + h * 64;
                if (ptx::elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t q_off = ((k / 4) * 16384 + (k % 4) * 32) >> 4, k_off = ((k / 4) * 1024 + (k % 4) * 32) >> 4;
                        ptx::mma_ss(col, dq + q_off, dk + k_off, g.idesc_s64, k > 0);
                    }
                    ptx::mma_commit(full);
                }
                __syncwarp();
            };
            // Rows of a V tile that hold nothing of the sequence (past its end, pages that are none): zeros,
            // as their weight is 0 and what lies there may be infinite.
            auto clear_rows = [&](uint32_t vslot, int left) {
                const unsigned absent = *(volatile unsigned *)&sh->absent[vslot];
                if (left >= kKeys && absent == 0) return;
                for (int r = lane; r < kKeys; r += 32)
                    if (r >= left || (absent >> (r >> 3) & 1)) clear_row<D>(ring + vslot * TB, r);
                ptx::fence_proxy_async_smem();
                __syncwarp();
            };
            // the stage of tile kt, past those before it, which are the other slot's
            auto take = [&](Ring<NR> &tiles, uint32_t first, int &pos, int kt, uint32_t &stage) -> bool {
                while (acquire(tiles, first, stage)) {
                    if (pos++ == kt) return true;
                    if (lane == 0) ptx::mbar_arrive(LSSAR_AT(kv_empty) + 8 * stage);
                }
                return false;
            };
            Item it;
            while (ok && next_item(it)) {
                release_item();
                const int step = it.step, begin = it.kt0 + (step == 2 ? w : 0);
                const bool live = begin < it.kt1;
                int kpos = it.kt0, vpos = it.kt0;
                uint32_t kslot, vslot;
                if (live) {
                    if (!(ok = wait_all(LSSAR_AT(q_full) + 8 * w, qs++ & 1, kErrQ))) break;
                    ptx::tc_fence_after();
                    if constexpr (PHASE == kStats) {
                        for (int kt = begin; ok && kt < it.kt1; kt += step) {
                            if (!(ok = take(keys, 0, kpos, kt, kslot)) || !(ok = issue_s(kslot))) break;
                            commit(LSSAR_AT(kv_empty) + 8 * kslot);
                        }
                    } else {
                        if (!(ok = take(keys, 0, kpos, begin, kslot))) break;
                        if constexpr (kSplit) {
                            issue_half(kslot, 0);
                            issue_half(kslot, 1);
                        } else {
                            if (!(ok = issue_s(kslot))) break;
                        }
                        commit(LSSAR_AT(kv_empty) + 8 * kslot);
                    }
                }
                if constexpr (PHASE == kValues) {
                    for (int kt = begin; ok && kt < it.kt1; kt += step) {
                        const bool next = kt + step < it.kt1;
                        if (next && !(ok = take(keys, 0, kpos, kt + step, kslot))) break;
                        if constexpr (kSepP) {
                            // the next scores as soon as the score warps have these
                            if (next && !(ok = issue_s(kslot))) break;
                            if (next) commit(LSSAR_AT(kv_empty) + 8 * kslot);
                        }
                        if (!(ok = take(values, NR, vpos, kt, vslot))) break;
                        clear_rows(vslot, it.len - kt * kKeys);
                        auto o_is_free = [&] {
                            return kt > begin || segs == 0 || wait_all(LSSAR_AT(o_free) + 8 * w, (segs - 1) & 1, kErrOFree);
                        };
                        if constexpr (kSplit) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                // this half's weights are in place of its scores
                                if (!(ok = wait_all(LSSAR_AT(s_free) + 16 * w + 8 * h, pv & 1, kErrSFree))) break;
                                if (h == 0 && !(ok = o_is_free())) break;
                                ptx::tc_fence_after();
                                issue_pv(vslot, 64 * h, 4, kt > begin || h > 0);
                                // (no scores follow the last tile's first half: a warp that raises its rows' reference waits for this)
                                if (kTurns && h == 0 && !next) commit(LSSAR_AT(p_free) + 8 * w);
                                // (before the commits that nothing waits for: each takes some 300 cycles)
                                if (next) issue_half(kslot, h);
                            }
                            if (!ok) break;
                        } else {
                            if (!(ok = wait_all(LSSAR_AT(p_full) + 8 * w, pv & 1, kErrPFull)) || !(ok = o_is_free())) break;
                            ptx::tc_fence_after();
                            issue_pv(vslot, 0, 8, kt > begin);
                            commit(LSSAR_AT(p_free) + 8 * w);
                        }
                        ++pv;
                        if (!next) {
                            commit(LSSAR_AT(o_full) + 8 * w);
                            ++segs;
                        }
                        commit(LSSAR_AT(kv_empty) + 8 * vslot);
                        if (!kSepP && next) commit(LSSAR_AT(kv_empty) + 8 * kslot);
                    }
                }
                // the last tiles may be the other slot's
                while (ok && kpos < it.kt1) {
                    if (!(ok = acquire(keys, 0, kslot))) break;
                    ++kpos;
                    if (lane == 0) ptx::mbar_arrive(LSSAR_AT(kv_empty) + 8 * kslot);
                }
                while (ok && PHASE == kValues && vpos < it.kt1) {
                    if (!(ok = acquire(values, NR, vslot))) break;
                    ++vpos;
                    if (lane == 0) ptx::mbar_arrive(LSSAR_AT(kv_empty) + 8 * vslot);
                }
            }
            __syncwarp();
        }
    } else {
        if constexpr (PHASE == kValues) ptx::setmaxnreg_inc<kScoreRegs>();
        // ------------------------------------------------------------ score warps
        const int wg = (warp - kScoreWarp0) >> 2, w = wg & 1, half = wg >> 1, quarter = warp & 3;
        const int in = quarter * 32 + lane;                      // row of the tile = TMEM lane
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_col = tmem + lane_addr + (PHASE == kStats ? w * 256 : w * kKeys) + half * 64;
        const uint32_t p_col = kSepP ? tmem + lane_addr + kPCol + 64 * w + 32 * half : s_col;
        const uint32_t o_col = tmem + lane_addr + kOCol + w * D + half * (D / 2);
        dcheck(tmem_in_range(s_col, tmem, 64, 512) && (PHASE == kStats || tmem_in_range(o_col, tmem, D / 2, 512)), err, kDbgTmem);
        const uint32_t s_full = LSSAR_AT(s_full) + 16 * w + (kSplit ? 8 * half : 0), s_free = LSSAR_AT(s_free) + 16 * w + (kSplit ? 8 * half : 0);
        const uint32_t p_done = (kSepP ? LSSAR_AT(p_full) + 8 * w : s_free), p_free = LSSAR_AT(p_free) + 8 * w;
        // this row's place in the exchange arrays, of the first parity, and the other half's
        const uint32_t mine = (w * 2 + half) * (kTileRows * 4) + 4 * in, others = (w * 2 + (half ^ 1)) * (kTileRows * 4) + 4 * in;
        constexpr uint32_t kParity = 4 * kTileRows * 4;
        constexpr float kMasked = MODE == kSigmoidRw ? INFINITY : -INFINITY;
        Ring<kSBufs> sb;
        uint32_t pv = 0, exchanges = 0, turns = 0, joints = 0;
        uint32_t own_segs = 0, other_segs = 0;                   // segments with this slot, with the other
        uint32_t tiles = 0;            // tiles of keys that the CTA has taken
        const int run = g.s.head->run;
        bool ok = true;
        auto field = [&](size_t offset) { return ptx::ld_shared_s32(LSSAR_AT(items) + items.slot() * (uint32_t)sizeof(Item) + (uint32_t)offset); };
#define LSSAR_ITEM(name) field(offsetof(Item, name))
        // The next segment's rows of q (any strides, any group): each thread half of its row, into the tile
        // that the last product of the segment before has read.  Returns whether this tile has any.
        auto gather = [&](uint32_t slot, bool &some) -> bool {
            if (!wait_all(LSSAR_AT(item_full) + 8 * (slot % kItems), slot / kItems & 1, kErrItem)) return false;
            some = gather_rows<D>(g, LSSAR_AT(items) + slot % kItems * (uint32_t)sizeof(Item), sq, w, half, in);
            return true;
        };
        // ... they are there; the normalised modes need their norms, whose halves meet next
        uint32_t meets = 0;
        auto hand_over = [&](bool some) {
            if (!some) return;
            asm volatile("cp.async.wait_all;" ::: "memory");
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(LSSAR_AT(q_full) + 8 * w);
            if constexpr (kNorm) {
                const uint32_t row = sq + w * TB + (D == 128 ? half * (kTileRows * 128) : 0) + in * 128;
                float s = 0.f;
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    uint4 u;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(row + (((D == 128 ? x : half * 4 + x) ^ (in & 7)) << 4)) : "memory");
                    s += squares(u, c.half);
                }
                ptx::st_shared_f32(LSSAR_AT(qq) + (meets & 1) * kParity + mine, s);
            }
        };
        // the two halves of this tile's rows have written what they exchange
        auto meet = [&] {
            ptx::mbar_arrive(LSSAR_AT(halves) + 8 * w);
            return wait_all(LSSAR_AT(halves) + 8 * w, meets++ & 1, kErrHalves);
        };
        // softmax: the exponents' offset for a reference (scores so large that their steps pass the room: without it)
        auto offset_of = [](float ref) {
            const float x = ref - Range16<MODE, HALF>::kRoom;
            return ref - x <= Range16<MODE, HALF>::kRoom ? x : ref;
        };
        bool some = false;
        ok = gather(0, some);
        if (ok) {
            hand_over(some);
            ok = meet();
        }
        // 32 products of the tile from column 32 x of this half on, as they are
        auto load = [&](uint32_t (&z)[32], uint32_t col) {
            ptx::tmem_ld32(col, z);
            ptx::tmem_ld_wait();
            ptx::reg_fence(z);
        };
        while (ok) {
            if (!wait_all(LSSAR_AT(item_full) + 8 * items.slot(), items.parity(), kErrItem)) break;
            const int kt0 = LSSAR_ITEM(kt0), kt1 = LSSAR_ITEM(kt1), rows = LSSAR_ITEM(rows), step = LSSAR_ITEM(step);
            if (kt0 < 0) break;
            // this slot's first tile, and its first row of the item
            const int begin = kt0 + (step - 1) * w, row0 = step == 1 ? w * kTileRows : 0;
            if (begin >= kt1) {                                  // nothing for this slot
                ++other_segs;
                tiles += kt1 - kt0;
                if ((ok = gather(items.i + 1, some))) {
                    hand_over(some);
                    ok = meet();
                }
                release_item();
                continue;
            }
            const bool live = rows > row0 + quarter * 32;
            const int v = min(row0 + in, rows - 1);              // row of the pair (past the last: the last)
            // last slot that the row attends to, and that of the warp's first row
            const int limit = LSSAR_ITEM(base) + LSSAR_ITEM(t0) + v / g.G;
            const int least = __shfl_sync(0xffffffffu, limit, 0);
            Row row = {};
            row.a = g.scale;
            if constexpr (kNorm) {
                const uint32_t at = LSSAR_AT(qq) + (meets - 1 & 1) * kParity;
                const float qq = ptx::ld_shared_f32(at + mine) + ptx::ld_shared_f32(at + others);
                row.a = g.scale * logf((float)(limit + 1)) / fmaxf(sqrtf(qq), 1e-12f);
            }
            int form = kMixed;
            if constexpr (PHASE == kValues && is_reweight(MODE)) {
                // the row's maximum and sum from the segments of its item
                float m = kLowest, s1 = 0.f;
                const int start = LSSAR_ITEM(start), each = tile_cost(rows), c0 = (start + each - 1) / run, c1 = (start + LSSAR_ITEM(nk) * each - 1) / run;
                const float2 *part = g.s.stats + (size_t)LSSAR_ITEM(item) * g.rows + v;
#pragma unroll 4
                for (int cta = c0; cta <= c1; ++cta) {
                    const float2 x = part[(size_t)cta * g.rows];
                    const float top = fmaxf(m, x.x);
                    s1 = MODE == kSoftmaxRw ? s1 * ptx::ex2(m - top) + x.y * ptx::ex2(x.x - top) : s1 + x.y;
                    m = top;
                }
                form = row_constants<MODE>(row, m, s1, limit + 1, a.p, g.exact_weights);
                // one form for the warp: all rows or none by one exponential
                const unsigned accurate = __ballot_sync(0xffffffffu, form == kAccurate), one = __ballot_sync(0xffffffffu, form == kOneExp);
                form = accurate ? kAccurate : one == 0xffffffffu ? kOneExp : kMixed;
            }
            if constexpr (PHASE == kValues && kOnePass) {
                row.ref = MODE == kSoftmax ? kLowest : kNoLift;
                row.x = MODE == kSoftmax ? kLowest : ptx::ex2(Range16<MODE, HALF>::kRoom - kNoLift);
                form = MODE == kLssa ? kAccurate : kMixed;
            }
            float m_run = MODE == kSigmoidRw ? INFINITY : MODE == kLssar ? kLowest : -INFINITY, sum_run = 0.f;
            float2 acc = make_float2(0.f, 0.f);
            for (int kt = begin; kt < kt1; kt += step) {
                const uint32_t buf = sb.slot(), col = s_col + buf * kKeys;
                if (!(ok = wait_all(s_full + 8 * buf, sb.parity(), kErrSFull))) break;
                ++sb.i;
                ptx::tc_fence_after();
                if (kt + step >= kt1) {
                    // the last product with this q is done (kSplit: the other half's too)
                    if (kSplit && !(ok = wait_all(LSSAR_AT(s_full) + 16 * w + 8 * (half ^ 1), (sb.i - 1) & 1, kErrSFull))) break;
                    if (!(ok = gather(items.i + 1, some))) break;
                }
                if (!live) {
                    // none of the item's rows: the barriers only
                    ptx::tc_fence_before();
                    if constexpr (PHASE == kStats || kSepP) ptx::mbar_arrive(s_free + 8 * buf);
                    if constexpr (PHASE == kValues) {
                        // (not before the last step's arrivals are all in, which its product follows)
                        if (kSepP && pv > 0 && !(ok = wait_all(p_free, (pv - 1) & 1, kErrPFree))) break;
                        ptx::mbar_arrive(p_done);
                        ++pv;
                    }
                    continue;
                }
                const uint32_t knorm = LSSAR_AT(knorm) + (tiles + (kt - kt0)) % kInfo * (kKeys * 4) + half * 256;
                const int last = limit - kt * kKeys - half * 64;      // last column of the half that is not masked
                const bool masked = least < kt * kKeys + half * 64 + 63;
                if constexpr (PHASE == kStats) {
                    if constexpr (MODE == kLssar) {
                        // Softplus by one exponential a score, in one block with the norms' products; again (rare), or
                        // under a mask, with the choice made for each 32 columns.
                        bool again = masked;
                        if (!masked) {
                            uint32_t r0[32], r1[32];
                            load(r0, col);
                            float2 sum = acc, prod[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)};
                            to_z<kNorm>(r0, knorm, row.a);
                            float top = max_of(r0, -INFINITY);
                            softplus_sum<false>(r0, sum, prod[0]);
                            load(r1, col + 32);
                            to_z<kNorm>(r1, knorm + 128, row.a);
                            top = max_of(r1, top);
                            softplus_sum<false>(r1, sum, prod[1]);
                            m_run = fmaxf(m_run, top);
                            again = __any_sync(0xffffffffu, top < 0.f);
                            if (!again) {
                                acc = sum;
                                sum_run += ptx::lg2((prod[0].x * prod[0].y) * (prod[1].x * prod[1].y));
                            }
                        }
                        if (again) {
#pragma unroll 1
                            for (int x = 0; x < 2; ++x) {
                                uint32_t z[32];
                                load(z, col + x * 32);
                                to_z<kNorm>(z, knorm + x * 128, row.a);
                                if (masked) mask(z, last - x * 32, kMasked);
                                const float top = max_of(z, -INFINITY);
                                m_run = fmaxf(m_run, top);
                                float2 prod = make_float2(1.f, 1.f);
                                if (__any_sync(0xffffffffu, top < 0.f)) {
                                    softplus_sum<true>(z, acc, prod);
                                } else {
                                    softplus_sum<false>(z, acc, prod);
                                    sum_run += ptx::lg2(prod.x * prod.y);
                                }
                            }
                        }
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(s_free + 8 * buf);           // the next product may write here
                        continue;
                    }
                    if constexpr (MODE == kSigmoidRw) {
                        const float2 one = make_float2(1.f, 1.f);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t z[32];
                            load(z, col + x * 32);
                            to_z<kNorm>(z, knorm + x * 128, row.a);
                            if (masked) mask(z, last - x * 32, kMasked);
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const float2 y = pair_at(z, j);
                                m_run = min3(m_run, y.x, y.y);
                                const float2 e = __fadd2_rn(make_float2(ptx::ex2(y.x), ptx::ex2(y.y)), one);
                                acc = __fadd2_rn(acc, make_float2(ptx::rcp(e.x), ptx::rcp(e.y)));
                            }
                        }
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(s_free + 8 * buf);
                        continue;
                    }
                    uint32_t r0[32], r1[32];
                    ptx::tmem_ld32(col, r0);
                    ptx::tmem_ld32(col + 32, r1);
                    ptx::tmem_ld_wait();
                    ptx::reg_fence(r0);
                    ptx::reg_fence(r1);
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(s_free + 8 * buf);               // the next product may write here
                    to_z<kNorm>(r0, knorm, row.a);
                    to_z<kNorm>(r1, knorm + 128, row.a);
                    if (masked) {
                        mask(r0, last, kMasked);
                        mask(r1, last - 32, kMasked);
                    }
                    if constexpr (MODE == kSoftmaxRw) tc::softmax_tile_stats(r0, r1, m_run, sum_run);
                    continue;
                }
                bool raise = false;
                float alpha = 1.f;
                if constexpr (kOnePass) {
                    // The reference of a row's weights: its running maximum (LSSA: up to 0, where softplus is
                    // at least 1), raised when a tile's passes it by more than the lag.  Both halves' maxima meet in
                    // shared memory.  A warp whose LSSA rows are all at 0 stays there.
                    if (MODE == kSoftmax || form == kAccurate) {
                        float top = -INFINITY;
#pragma unroll 1
                        for (int x = 0; x < 2; ++x) {
                            uint32_t z[32];
                            load(z, col + x * 32);
                            if constexpr (MODE == kLssa) to_z<true>(z, knorm + x * 128, row.a);
                            if (masked) mask(z, last - x * 32, -INFINITY);
                            top = max_of(z, top);
                        }
                        if constexpr (MODE == kSoftmax) top = __fmul_rn(top, row.a);      // (rounded as the scores are, in no FMA)
                        if (kTurns && kt > begin) {
                            if (!(ok = wait_all(LSSAR_AT(turn) + 64 * (half ^ 1) + 32 * w + 8 * quarter, (turns - (half ^ 1)) & 1, kErrTileMax))) break;
                            const float ref = ptx::ld_shared_f32(LSSAR_AT(tmax) + kParity + others), x = offset_of(ref);
                            const float f = ptx::ex2(row.x - x);
                            acc = __fmul2_rn(acc, make_float2(f, f));
                            row.x = x;
                            row.ref = ref;
                        } else {
                            const uint32_t at = LSSAR_AT(tmax) + (kTurns ? 0u : (exchanges & 1) * kParity);     // (kTurns: references in the other)
                            ptx::st_shared_f32(at + mine, top);
                            // (LSSA in halves: half 0 learns here that the last tile's second product, which half 1's
                            // scores followed, has left O)
                            if constexpr (kSplit) ptx::tc_fence_before();
                            ptx::mbar_arrive(LSSAR_AT(tile_max) + 32 * w + 8 * quarter);
                            if (!(ok = wait_all(LSSAR_AT(tile_max) + 32 * w + 8 * quarter, exchanges & 1, kErrTileMax))) break;
                            if constexpr (kSplit) ptx::tc_fence_after();
                            top = fmaxf(top, ptx::ld_shared_f32(at + others));
                            ++exchanges;
                        }
                        if constexpr (MODE == kLssa) top = fminf(top, 0.f);
                        raise = top - row.ref > Range16<MODE, HALF>::kLag || (MODE == kLssa && top >= 0.f && row.ref < 0.f);
                        if (raise) {
                            if constexpr (MODE == kSoftmax) {
                                const float x = offset_of(top);
                                alpha = ptx::ex2(row.x - x);
                                row.x = x;
                            } else {
                                alpha = ptx::ex2(row.ref - top);
                                row.x = ptx::ex2(Range16<MODE, HALF>::kRoom - top);
                            }
                            row.ref = top;
                            acc = __fmul2_rn(acc, make_float2(alpha, alpha));
                        }
                        if constexpr (kTurns) {
                            ptx::st_shared_f32(LSSAR_AT(tmax) + kParity + mine, row.ref);
                            ptx::mbar_arrive(LSSAR_AT(turn) + 64 * half + 32 * w + 8 * quarter);
                            ++turns;
                        }
                        if constexpr (MODE == kLssa) form = __all_sync(0xffffffffu, row.ref >= 0.f) ? kMixed : kAccurate;
                        if constexpr (MODE == kSoftmax) form = __any_sync(0xffffffffu, fabsf(row.ref) > 65536.f) ? kAccurate : kMixed;
                    }
                }
                // P and O are free once the product before has read the one and written the other
                auto free_p = [&] {
                    if constexpr (!kSepP) return true;
                    if (pv == 0) return true;
                    if (!wait_all(p_free, (pv - 1) & 1, kErrPFree)) return false;
                    ptx::tc_fence_after();
                    return true;
                };
                auto free_s = [&] {                                   // the next product may write here
                    if constexpr (kSepP) {
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(s_free);
                    }
                };
                if (masked) {
#pragma unroll 1
                    for (int x = 0; ok && x < 2; ++x) {
                        uint32_t z[32], pk[16];
                        load(z, col + x * 32);
                        if (x == 1) free_s();
                        if constexpr (MODE != kSoftmax) to_z<kNorm>(z, knorm + x * 128, row.a);
                        mask(z, last - x * 32, kMasked);
                        with_form<MODE>(form, g.power.exact, [&](auto f) {
                            weights16<MODE, HALF, f.kForm, f.kP>(z, 0, row, g.power, acc, pk);
                            weights16<MODE, HALF, f.kForm, f.kP>(z + 16, 8, row, g.power, acc, pk + 8);
                            return true;
                        });
                        if (x == 0 && !(ok = free_p())) break;
                        ptx::tmem_st16(p_col + x * 16, pk);
                    }
                } else {
                    ok = with_form<MODE>(form, g.power.exact, [&](auto f) {
#pragma unroll 1
                        for (int x = 0; x < 2; ++x) {
                            uint32_t z[32], pk[16];
                            load(z, col + x * 32);
                            if (x == 1) free_s();
                            if constexpr (MODE != kSoftmax) to_z<kNorm>(z, knorm + x * 128, row.a);
                            weights16<MODE, HALF, f.kForm, f.kP>(z, 0, row, g.power, acc, pk);
                            weights16<MODE, HALF, f.kForm, f.kP>(z + 16, 8, row, g.power, acc, pk + 8);
                            if (x == 0 && !free_p()) return false;
                            ptx::tmem_st16(p_col + x * 16, pk);
                        }
                        return true;
                    });
                }
                if (!ok) break;
                if constexpr (kOnePass) {
                    if (kt > begin && __any_sync(0xffffffffu, raise)) {
                        if constexpr (kTurns) {
                            // the product of the turn before is done: the other half's next scores follow it
                            const bool next = kt + step < kt1;
                            const uint32_t bar = half == 0 || next ? LSSAR_AT(s_full) + 16 * w + 8 * (half ^ 1) : LSSAR_AT(p_free) + 8 * w;
                            if (!(ok = wait_all(bar, (half == 0 ? sb.i - 1 : next ? sb.i : own_segs) & 1, kErrSFull))) break;
                            ptx::tc_fence_after();
                        }
                        const uint32_t first = kTurns ? tmem + lane_addr + kOCol + w * D : o_col;
#pragma unroll 1
                        for (int x = 0; x < (kTurns ? D : D / 2); x += 16) {
                            uint32_t o[16];
                            ptx::tmem_ld16(first + x, o);
                            ptx::tmem_ld_wait();
                            ptx::reg_fence(o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                            ptx::tmem_st16(first + x, o);
                        }
                    }
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                if constexpr (kSplit && MODE == kLssa) {
                    // (the first half's product must not start while the other half's columns of O are rescaled)
                    if (kt > begin && __any_sync(0xffffffffu, raise)) {
                        ptx::mbar_arrive(LSSAR_AT(tile_max) + 32 * w + 8 * quarter);
                        if (!(ok = wait_all(LSSAR_AT(tile_max) + 32 * w + 8 * quarter, exchanges++ & 1, kErrTileMax))) break;
                        ptx::tc_fence_after();           // (the other half's stores come before this arrival too)
                        ptx::tc_fence_before();
                    }
                }
                ptx::mbar_arrive(p_done);
                ++pv;
            }
            if (!ok) break;
            tiles += kt1 - kt0;
            hand_over(some);
            // the two halves of a row meet
            const uint32_t par = meets & 1;
            float part = (acc.x + acc.y) + sum_run;
            ptx::st_shared_f32(LSSAR_AT(s) + par * kParity + mine, part);
            const float m_part = MODE == kSigmoidRw ? -m_run : fmaxf(m_run, kLowest);
            if constexpr (PHASE == kStats) ptx::st_shared_f32(LSSAR_AT(m) + par * kParity + mine, m_part);
            if constexpr (kTurns) ptx::st_shared_f32(LSSAR_AT(m) + par * kParity + mine, row.x);
            if (!(ok = meet())) break;
            float other = ptx::ld_shared_f32(LSSAR_AT(s) + par * kParity + others);
            const bool valid = row0 + in < rows;
            // Two slots with the same rows: the first adds the second's part to its own.
            const bool both = step == 2 && kt0 + 1 < kt1, second = both && w == 1;
            const uint32_t joint_at = (joints & 1) * (2 * kTileRows * 4) + 8 * in;
            auto join = [&](float x, float y) -> bool {           // the second's pair of values in place, or there
                if (second) {
                    if (joints > 0 && !wait_all(LSSAR_AT(joint), (joints - 1) & 1, kErrJoint)) return false;
                    if (half == 0) {
                        ptx::st_shared_f32(LSSAR_AT(other) + joint_at, x);
                        ptx::st_shared_f32(LSSAR_AT(other) + joint_at + 4, y);
                    }
                }
                ptx::mbar_arrive(LSSAR_AT(joint));
                return second || wait_all(LSSAR_AT(joint), joints & 1, kErrJoint);
            };
            if constexpr (PHASE == kStats) {
                if (half == 0) {
                    const float m1 = ptx::ld_shared_f32(LSSAR_AT(m) + par * kParity + others);
                    float m = fmaxf(m_part, m1), s = MODE == kSoftmaxRw ? part * ptx::ex2(m_part - m) + other * ptx::ex2(m1 - m) : part + other;
                    if (both) {
                        if (!(ok = join(m, s))) break;
                        const float mo = ptx::ld_shared_f32(LSSAR_AT(other) + joint_at), so = ptx::ld_shared_f32(LSSAR_AT(other) + joint_at + 4);
                        const float top = fmaxf(m, mo);
                        s = MODE == kSoftmaxRw ? s * ptx::ex2(m - top) + so * ptx::ex2(mo - top) : s + so;
                        m = top;
                        ++joints;
                    }
                    const long long at = LSSAR_ITEM(item) + (long long)blockIdx.x;
                    if (valid && !second && dcheck(v < g.rows, err, kDbgGlobal)) g.s.stats[at * g.rows + v] = make_float2(m, s);
                }
                release_item();
                continue;
            }
            if constexpr (kTurns) {
                // the last turn's reference, half 1's, holds for both
                const float x = ptx::ld_shared_f32(LSSAR_AT(m) + par * kParity + others);
                if (half == 0) {
                    part *= ptx::ex2(row.x - x);
                    row.x = x;
                } else {
                    other *= ptx::ex2(x - row.x);
                }
            }
            // (half 0's part first in both, so that both see the same sum)
            float sum = half == 0 ? part + other : other + part;
            if (limit >= LSSAR_ITEM(first_bad)) sum = NAN;
            float ref = MODE == kSoftmax ? row.x : row.ref, f = 1.f, fo = 0.f;      // the parts' factors
            if (both) {
                if (!(ok = join(ref, sum))) break;
                fo = 1.f;
                if (!second) {
                    const float ro = ptx::ld_shared_f32(LSSAR_AT(other) + joint_at), so = ptx::ld_shared_f32(LSSAR_AT(other) + joint_at + 4);
                    if constexpr (kOnePass) {
                        const float top = fmaxf(ref, ro);
                        f = ptx::ex2(ref - top);
                        fo = ptx::ex2(ro - top);
                        ref = top;
                    }
                    sum = sum * f + so * fo;
                }
                ++joints;
            }
            if (!second) {
                if (!(ok = wait_all(LSSAR_AT(o_full) + 8 * w, own_segs & 1, kErrOFull))) break;
                if (both && !(ok = wait_all(LSSAR_AT(o_full) + 8 * (w ^ 1), other_segs & 1, kErrOFull))) break;
            }
            ++own_segs;
            if (step == 1 || both) ++other_segs;
            if (second) {
                release_item();
                continue;
            }
            ptx::tc_fence_after();
            const int b = LSSAR_ITEM(b), hq = LSSAR_ITEM(h) * g.G + v % g.G, t = LSSAR_ITEM(t0) + v / g.G;
            const bool whole = kt0 == 0 && kt1 == LSSAR_ITEM(nk);
            // a segment's part: of the run's first item in its first place, of its last in its second
            const int place = 2 * blockIdx.x + (kt0 == 0 ? 1 : 0);
            const size_t to = (size_t)place * g.rows + v;
            const bool in_range = dcheck(b < c.B && hq < a.H && t < a.n && v < g.rows && place < 2 * g.ctas, err, kDbgGlobal);
            const float inv = 1.f / sum;
            if (valid && in_range && !whole && half == 0) g.s.sums[to] = make_float2(ref, sum);
            if (live) {
#pragma unroll 1
                for (int x = 0; x < D / 64; ++x) {
                    uint32_t o[32];
                    load(o, o_col + x * 32);
                    if (both) {
                        uint32_t p[32];
                        load(p, o_col + D + x * 32);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f + __uint_as_float(p[j]) * fo);
                    }
                    if (!valid || !in_range) continue;
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (((size_t)b * a.H + hq) * a.n + t) * D + half * (D / 2) + x * 32);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t u[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 f = __fmul2_rn(pair_at(o, 8 * j + 2 * k), make_float2(inv, inv));
                                u[k] = HALF ? ptx::pack_f16x2(f.x, f.y) : ptx::pack_bf16x2(f.x, f.y);
                            }
                            dst[j] = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(g.s.o + to * D + half * (D / 2) + x * 32);
#pragma unroll
                        for (int j = 0; j < 8; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                }
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(LSSAR_AT(o_free) + 8 * w);
            if (both) ptx::mbar_arrive(LSSAR_AT(o_free) + 8 * (w ^ 1));
            release_item();
        }
#undef LSSAR_ITEM
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- join

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;

// Items that lie in several runs: block x takes the one that run x + 1 begins inside of, if that is
// the first such run; blockIdx.y: a group of its rows.
template <int D, bool HALF, bool RELATIVE>
__global__ void __launch_bounds__(kJoinThreads) attend_join(const __grid_constant__ Args g) {
    const PagedAttend &a = g.a;
    const PagedCache &c = a.c;
    const Header head = *g.s.head;             // the plan is there (see attend_kernel)
    const int cta = blockIdx.x + 1;
    const long long x = (long long)cta * head.run;
    bool some = x < head.total;
    int4 en = make_int4(0, 0, 1, 0);
    int h = 0, last = 0, rows = 0, t0 = 0;
    if (some) {
        en = g.s.first[2 * cta];
        h = (int)(x - en.w) / en.z;
        t0 = en.y * g.tokens;
        rows = rows_of_pair(g, g.s.first[2 * cta + 1].y, t0);
        // the runs of its first and last tile
        const int each = tile_cost(rows), start = en.w + h * en.z + kItemCost;
        last = (en.w + (h + 1) * en.z - 1) / head.run;
        some = (start + each - 1) / head.run == cta - 1 && last >= cta;
    }
    ptx::grid_dependency_wait();               // the segments' parts too (in every block: the call's end waits for them)
    if (!some) return;
    constexpr int kLanes = D / 4, kStep = kJoinThreads / kLanes;
    const int part = threadIdx.x % kLanes;
#pragma unroll 1
    for (int r = blockIdx.y * kJoinRows + threadIdx.x / kLanes; r < min(rows, (int)(blockIdx.y + 1) * kJoinRows); r += kStep) {
        float m = RELATIVE ? kLowest : 0.f, w = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = cta - 1; k <= last; ++k) {
            const size_t at = (size_t)(2 * k + (k == cta - 1)) * g.rows + r;      // its first segment in the second place
            const float2 s = g.s.sums[at];
            const float4 v = reinterpret_cast<const float4 *>(g.s.o + at * D)[part];
            float f = 1.f;
            if (RELATIVE) {
                const float top = fmaxf(m, s.x), old = ptx::ex2(m - top);
                f = ptx::ex2(s.x - top);
                m = top;
                w *= old;
                o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
            }
            w = fmaf(s.y, f, w);
            o = make_float4(fmaf(v.x, f, o.x), fmaf(v.y, f, o.y), fmaf(v.z, f, o.z), fmaf(v.w, f, o.w));
        }
        const int tok = r / g.G, hq = h * g.G + r - tok * g.G;
        const float inv = 1.f / w;
        const uint32_t lo = HALF ? ptx::pack_f16x2(o.x * inv, o.y * inv) : ptx::pack_bf16x2(o.x * inv, o.y * inv);
        const uint32_t hi = HALF ? ptx::pack_f16x2(o.z * inv, o.w * inv) : ptx::pack_bf16x2(o.z * inv, o.w * inv);
        const size_t out_row = ((size_t)en.x * a.H + hq) * a.n + t0 + tok;
        if (dcheck(en.x < c.B && hq < a.H && t0 + tok < a.n, c.err, kDbgGlobal))
            reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + out_row * D)[part] = make_uint2(lo, hi);
    }
}

// ---------------------------------------------------------------- launches

template <int D, int MODE, bool HALF, int PHASE>
cudaError_t launch_phase(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, cudaStream_t stream) {
    static PerDeviceOnce once;
    const void *fn = (const void *)attend_kernel<D, MODE, HALF, PHASE>;
    constexpr int smem = Cfg<D>::kSmem;
    const cudaError_t e = per_device_once(once, nullptr, [&](int &) {
        // registers move between the warpgroups (kValues): only a launch at exactly
        // kLaunchRegs a thread adds up
        cudaFuncAttributes attr;
        const cudaError_t x = cudaFuncGetAttributes(&attr, fn);
        if (x != cudaSuccess) return x;
        if (PHASE == kValues && attr.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    void *args[] = {(void *)&km, (void *)&vm, (void *)&g};
    return paged::launch_kernel(fn, g.ctas, kThreads, smem, true, args, stream);
}

template <int D, int MODE, bool HALF>
cudaError_t launch_mode(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t stream) {
    int norms = uses_normalised_qk(MODE);
    void *prep[] = {(void *)&g, (void *)&norms};
    cudaError_t e = paged::launch_kernel((const void *)attend_prepare<D>, norms ? 1 + 4 * sms : 1, kPrepThreads, 0, false, prep, stream);
    if (e != cudaSuccess) return e;
    if constexpr (is_reweight(MODE))
        if ((e = launch_phase<D, MODE, false, kStats>(km, vm, g, stream)) != cudaSuccess) return e;
    if ((e = launch_phase<D, MODE, HALF, kValues>(km, vm, g, stream)) != cudaSuccess) return e;
    if (g.ctas < 2) return cudaSuccess;
    void *args[] = {(void *)&g};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)g.ctas - 1, (unsigned)(g.rows + kJoinRows - 1) / kJoinRows);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, (const void *)attend_join<D, HALF, !is_reweight(MODE)>, args);
}

// One call per mode and d, in files of their own so that the instances compile in parallel.
using Launch = cudaError_t(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t st);
Launch softmax_d64, softmax_d128, lssa_d64, lssa_d128, lssar_d64, lssar_d128, softmax_rw_d64, softmax_rw_d128, sigmoid_rw_d64, sigmoid_rw_d128;

#define LSSAR_ATTEND_INSTANCE(NAME, MODE, D)                                                                             \
    cudaError_t NAME(const CUtensorMap &km, const CUtensorMap &vm, const Args &g, int sms, cudaStream_t st) {            \
        return g.a.c.half ? launch_mode<D, MODE, true>(km, vm, g, sms, st) : launch_mode<D, MODE, false>(km, vm, g, sms, st); \
    }

}  // namespace attend
}  // namespace lssar
