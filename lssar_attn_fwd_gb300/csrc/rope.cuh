// Rotary positions: internal declarations.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "lssar_attn_fwd.h"
#include "paged.cuh"

namespace lssar {

constexpr int kMaxPairs = 64;   // rot_dim / 2

// The turn of every pair, in turns per position as a 64-bit fraction: the phase of
// position m is m * turn[c] modulo 2^64, exact for every 32-bit m.  The table's own
// rounding, of doubles, is below 2^-50 turns per position: of a frequency f <= 1 it is at most
// 5 |ln f| x 2^-53 by the exponent (f |ln f| <= 1 / e) and 25 x 2^-53 by exp(), the products and 2 pi, over 2 pi.
// It grows to 2^-19 turns at m = 2^31 (found: 2^-24 at a base of 10000, 2^-22 at the worst of 207 bases).
// fp32 angles would be off by 0.06 radians at a position of 10^6.
struct RotaryTable {
    unsigned long long turn[kMaxPairs];
    int rot;             // elements that turn
    bool interleaved;
};

// Checks the description for heads of d elements and fills the table; LSSAR_OK or an error.
int rotary_table(const lssar_rotary_t *r, int d, RotaryTable *out);

// One tensor that turns: rows of (b, h, t) by element strides.
struct RopeView {
    const uint16_t *x;
    uint16_t *y;
    long long xs[3], ys[3];
    int H;
};

struct Rope {
    RopeView v[2];       // q, k (H = 0: none)
    RotaryTable table;
    int B, L, d;
    bool half, back;
    const int *positions;
    int per_token;
};
cudaError_t launch_rope(const Rope &pr, cudaStream_t stream);

struct PagedAppendRope {
    PagedAppend a;
    RopeView q;
    RotaryTable table;
};
cudaError_t launch_paged_append_rope(const PagedAppendRope &pr, cudaStream_t stream);

}  // namespace lssar
