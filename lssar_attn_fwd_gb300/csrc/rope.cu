// Rotary positions: queries and keys of a training step (forward and gradients), and the
// paged append that turns queries and keys on their way.
//
// Pair c of a row at position m, (u, v) -> (u cos a - v sin a, u sin a + v cos a) with
// a = m f_c; the gradient turns back (-a).  2d bytes of each row are read and as many
// written, a few operations an element, so HBM bounds it.  A thread takes 16 elements of a
// row (eight pairs, two 16-byte pieces: the pieces u and u + rot/16 of a half layout, 2u and
// 2u + 1 of an interleaved one), so that it works out eight sines and cosines once per token and
// keeps them in registers over the heads of its group.
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rope.cuh"
#include "api_checks.cuh"
#include "tc_host.cuh"
#include "tc_ptx.cuh"

namespace lssar {

int rotary_table(const lssar_rotary_t *r, int d, RotaryTable *out) {
    if (!r) return LSSAR_ERR_NULL;
    const int rot = r->rot_dim;
    if (!(r->base > 1.0) || !std::isfinite(r->base) || rot < 16 || rot > d || rot % 16 || r->scaling < LSSAR_ROPE_PLAIN ||
        r->scaling > LSSAR_ROPE_BANDS || (r->interleaved != 0 && r->interleaved != 1))
        return LSSAR_ERR_ROTARY;
    if (r->scaling != LSSAR_ROPE_PLAIN && (!(r->factor >= 1.0) || !std::isfinite(r->factor))) return LSSAR_ERR_ROTARY;
    if (r->scaling == LSSAR_ROPE_BANDS &&
        (!(r->low >= 0.0) || !(r->high > r->low) || !std::isfinite(r->high) || r->original_length < 1))
        return LSSAR_ERR_ROTARY;
    const double two_pi = 6.283185307179586476925;
    const double base = r->scaling == LSSAR_ROPE_BASE ? r->base * std::pow(r->factor, (double)rot / (rot - 2)) : r->base;
    if (!std::isfinite(base)) return LSSAR_ERR_ROTARY;
    for (int c = 0; c < kMaxPairs; ++c) out->turn[c] = 0;
    // by exp() for every eighth pair, and products between (at most 7 x 3 x 2^-53 of each)
    const double step = -2.0 / rot * std::log(base), ratio = std::exp(step);
    double g = 1.0;
    for (int c = 0; c < rot / 2; ++c) {
        g = c % 8 == 0 ? std::exp(step * c) : g * ratio;
        double f = g;
        if (r->scaling == LSSAR_ROPE_LINEAR) f /= r->factor;
        if (r->scaling == LSSAR_ROPE_BANDS) {
            const double keep = std::fmin(1.0, std::fmax(0.0, (r->original_length * f / two_pi - r->low) / (r->high - r->low)));
            f *= keep + (1.0 - keep) / r->factor;
        }
        out->turn[c] = (unsigned long long)std::ldexp(f / two_pi, 64);   // f <= 1: below 2^64
    }
    out->rot = rot;
    out->interleaved = r->interleaved != 0;
    return LSSAR_OK;
}

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;   // heads whose loads are in flight together

template <typename T>
struct Pack;
template <>
struct Pack<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t x) {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float2 x) { return ptx::pack_bf16x2(x.x, x.y); }
};
template <>
struct Pack<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }
    static __device__ __forceinline__ uint32_t pack(float2 x) { return ptx::pack_f16x2(x.x, x.y); }
};

// The pieces of 8 elements that a thread takes of every row, and its pairs' cosines and sines.
struct Turn {
    float c[8], s[8];
    int first, second;   // pieces
    bool turns;          // else they are copied
};

__device__ __forceinline__ Turn make_turn(const RotaryTable &t, int unit, long long pos, bool back) {
    Turn r;
    const int units = t.rot / 16;
    r.turns = unit < units;
    const bool split = r.turns && !t.interleaved;
    r.first = split ? unit : 2 * unit;
    r.second = split ? unit + units : 2 * unit + 1;
    if (r.turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the high word of the phase, as a signed fraction of half a turn
            const unsigned long long phase = (unsigned long long)pos * t.turn[unit * 8 + i];
            const float a = (float)(int)(phase >> 32) * 4.656612873077393e-10f;   // 2^-31
            sincospif(a, &r.s[i], &r.c[i]);
            if (back) r.s[i] = -r.s[i];
        }
    }
    return r;
}

// Eight pairs: in a half layout pair i is (x0[i], x1[i]); interleaved, x0 holds pairs 0-3, x1 4-7.
template <typename T, bool INTER>
__device__ __forceinline__ void turn_pairs(uint4 &x0, uint4 &x1, const Turn &t) {
    uint32_t *a = reinterpret_cast<uint32_t *>(&x0), *b = reinterpret_cast<uint32_t *>(&x1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 u = Pack<T>::unpack(a[i]), v = Pack<T>::unpack(b[i]);
        if (INTER) {
            u = make_float2(u.x * t.c[i] - u.y * t.s[i], u.x * t.s[i] + u.y * t.c[i]);
            v = make_float2(v.x * t.c[i + 4] - v.y * t.s[i + 4], v.x * t.s[i + 4] + v.y * t.c[i + 4]);
        } else {
            const float2 c = make_float2(t.c[2 * i], t.c[2 * i + 1]), s = make_float2(t.s[2 * i], t.s[2 * i + 1]);
            const float2 w = u;
            u = make_float2(w.x * c.x - v.x * s.x, w.y * c.y - v.y * s.y);
            v = make_float2(w.x * s.x + v.x * c.x, w.y * s.y + v.y * c.y);
        }
        a[i] = Pack<T>::pack(u);
        b[i] = Pack<T>::pack(v);
    }
}

// Heads [h0, h1) of one token: from x + h * xs to y + h * ys, turned (or copied, TURN false).
template <typename T, bool INTER, bool TURN>
__device__ __forceinline__ void turn_heads(const uint16_t *x, long long xs, uint16_t *y, long long ys, int h0, int h1, const Turn &t) {
#pragma unroll 1
    for (int h = h0; h < h1; h += kAtOnce) {
        uint4 a[kAtOnce], b[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
            if (h + e < h1) {
                const uint4 *row = reinterpret_cast<const uint4 *>(x + (h + e) * xs);
                a[e] = row[t.first];
                b[e] = row[t.second];
            }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
            if (h + e < h1) {
                if (TURN && t.turns) turn_pairs<T, INTER>(a[e], b[e], t);
                uint4 *row = reinterpret_cast<uint4 *>(y + (h + e) * ys);
                row[t.first] = a[e];
                row[t.second] = b[e];
            }
    }
}

// blockIdx.y: a group of `group` heads of the heads of q, then of k.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_rows(const __grid_constant__ Rope r, int group) {
    const int units = r.d / 16, unit = threadIdx.x % units;
    const long long token = (long long)blockIdx.x * (kThreads / units) + threadIdx.x / units;
    if (token >= (long long)r.B * r.L) return;
    const int b = (int)(token / r.L), t = (int)(token - (long long)b * r.L);
    long long pos = t;
    if (r.positions) pos = r.per_token ? r.positions[token] : (long long)r.positions[b] + t;
    const Turn turn = make_turn(r.table, unit, pos, r.back);
    const int g0 = blockIdx.y * group, g1 = min(g0 + group, r.v[0].H + r.v[1].H);
    int base = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const RopeView &v = r.v[i];
        const int h0 = max(g0 - base, 0), h1 = min(g1 - base, v.H);
        base += v.H;
        // what does not turn is where it should be already when the call is in place
        if (h0 >= h1 || (v.x == v.y && !turn.turns)) continue;
        turn_heads<T, INTER, true>(v.x + b * v.xs[0] + t * v.xs[2], v.xs[1], v.y + b * v.ys[0] + t * v.ys[2], v.ys[1], h0, h1, turn);
    }
}

// blockIdx.y: a group of `group` heads of the heads of q, then of k, then of v.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) append_rope_rows(const __grid_constant__ PagedAppendRope r, int group) {
    const PagedAppend &a = r.a;
    const PagedCache &c = a.c;
    const int units = c.d / 16, unit = threadIdx.x % units;
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x, token = id / units;
    if (blockIdx.y == 0 && id < c.B) {
        const int len = c.lens[id], cnt = a.counts ? a.counts[id] : a.n;
        const bool ok = len >= 0 && cnt >= 0 && cnt <= a.n && (long long)len + cnt <= c.capacity();
        if (!ok) atomicCAS(c.err, 0u, (unsigned)kErrPagedLength);
        a.lens_out[id] = ok ? len + cnt : len;
    }
    if (token >= (long long)c.B * a.n) return;
    const int b = (int)(token / a.n), t = (int)(token - (long long)b * a.n);
    const int len = c.lens[b], cnt = a.counts ? a.counts[b] : a.n;
    const int g0 = blockIdx.y * group, g1 = min(g0 + group, r.q.H + 2 * c.Hkv);
    const RopeView &q = r.q;
    if (len < 0 || cnt < 0 || cnt > a.n || (long long)len + cnt > c.capacity()) {
        // left alone; without counts its rows of q are asked for all the same, and nothing may stay unwritten
        if (a.counts || q.x == q.y) return;
        for (int h = g0; h < min(g1, q.H); ++h) {
            uint4 *row = reinterpret_cast<uint4 *>(q.y + b * q.ys[0] + h * q.ys[1] + t * q.ys[2]);
            row[2 * unit] = row[2 * unit + 1] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    if (t >= cnt) return;
    const long long first = a.first ? a.first[b] : len;
    const int slot = len + t, i = slot / c.page_size, row = slot - i * c.page_size;
    const int page = c.table[(size_t)b * c.max_pages + i];
    const bool known = (unsigned)page < (unsigned)c.n_pages;
    if (blockIdx.y == 0) {
        for (int h = unit; h < c.Hkv; h += units) {
            const size_t at = ((size_t)b * c.Hkv + h) * c.capacity() + slot;
            if (a.scores) a.scores[at] = 0.f;
            if (a.positions) a.positions[at] = (int)(first + t);
        }
        if (!known && unit == 0) atomicCAS(c.err, 0u, (unsigned)kErrPagedPage);
    }
    const Turn turn = make_turn(r.table, unit, first + t, false);
    if (g0 < q.H && (q.x != q.y || turn.turns))
        turn_heads<T, INTER, true>(q.x + b * q.xs[0] + t * q.xs[2], q.xs[1], q.y + b * q.ys[0] + t * q.ys[2], q.ys[1], g0, min(g1, q.H), turn);
    if (!known || !dcheck(row >= 0 && row < c.page_size, c.err, kDbgGlobal)) return;
    const size_t to = page * c.page_stride + (size_t)row * c.d;
    const long long per_head = (long long)c.page_size * c.d;
    int h0 = max(g0 - q.H, 0), h1 = min(g1 - q.H, c.Hkv);
    turn_heads<T, INTER, true>(static_cast<const uint16_t *>(a.k_new) + b * a.ks[0] + t * a.ks[2], a.ks[1],
                               static_cast<uint16_t *>(c.k) + to, per_head, h0, h1, turn);
    h0 = max(g0 - q.H - c.Hkv, 0), h1 = min(g1 - q.H - c.Hkv, c.Hkv);
    turn_heads<T, INTER, false>(static_cast<const uint16_t *>(a.v_new) + b * a.vs[0] + t * a.vs[2], a.vs[1],
                                static_cast<uint16_t *>(c.v) + to, per_head, h0, h1, turn);
}

// Heads per block, at most 8: as many as leave four blocks per SM, so that sines are worked out seldom.
// (8 sequences of 1K tokens, 24 heads of 64: 3 heads 12.9 us, 2 heads 14.6, 1 head 21; 4 of 4K, 32 heads of
// 128: 8 heads 42.0 us, 16 heads 45.7, 32 heads 50.)
int heads_per_block(long long token_blocks, int heads, int sms) {
    int group = heads;
    while (group > 1 && (group > 8 || token_blocks * ((heads + group - 1) / group) < 4LL * sms)) group = (group + 1) / 2;
    while ((heads + group - 1) / group > 65535) group *= 2;
    return group;
}

}  // namespace

cudaError_t launch_rope(const Rope &pr, cudaStream_t stream) {
    int sms = 0;
    const cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return e;
    const int rows = kThreads / (pr.d / 16), heads = pr.v[0].H + pr.v[1].H;
    const long long blocks = ((long long)pr.B * pr.L + rows - 1) / rows;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int group = heads_per_block(blocks, heads, sms);
    const dim3 grid((unsigned)blocks, (heads + group - 1) / group);
    const bool inter = pr.table.interleaved;
    if (pr.half) {
        if (inter) rope_rows<__half, true><<<grid, kThreads, 0, stream>>>(pr, group);
        else rope_rows<__half, false><<<grid, kThreads, 0, stream>>>(pr, group);
    } else {
        if (inter) rope_rows<__nv_bfloat16, true><<<grid, kThreads, 0, stream>>>(pr, group);
        else rope_rows<__nv_bfloat16, false><<<grid, kThreads, 0, stream>>>(pr, group);
    }
    return cudaGetLastError();
}

cudaError_t launch_paged_append_rope(const PagedAppendRope &pr, cudaStream_t stream) {
    PagedAppendRope r = pr;
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return e;
    if ((e = error_word_ptr(&r.a.c.err)) != cudaSuccess) return e;
    const int units = r.a.c.d / 16, heads = r.q.H + 2 * r.a.c.Hkv;
    const long long threads = (long long)r.a.c.B * r.a.n * units, least = r.a.c.B;
    const long long blocks = ((threads > least ? threads : least) + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int group = heads_per_block(blocks, heads, sms);
    const dim3 grid((unsigned)blocks, (heads + group - 1) / group);
    const bool inter = r.table.interleaved;
    if (r.a.c.half) {
        if (inter) append_rope_rows<__half, true><<<grid, kThreads, 0, stream>>>(r, group);
        else append_rope_rows<__half, false><<<grid, kThreads, 0, stream>>>(r, group);
    } else {
        if (inter) append_rope_rows<__nv_bfloat16, true><<<grid, kThreads, 0, stream>>>(r, group);
        else append_rope_rows<__nv_bfloat16, false><<<grid, kThreads, 0, stream>>>(r, group);
    }
    return cudaGetLastError();
}

namespace {

int rope_call(const void *q, const long long *qs, void *q_out, int H, const void *k, const long long *ks, void *k_out, int Hk,
              int B, int L, int d, int dtype, const lssar_rotary_t *rotary, const int *positions, int per_token, bool back,
              cudaStream_t stream) {
    if (!q || !qs || !q_out || (k && (!ks || !k_out))) return LSSAR_ERR_NULL;
    if (d != 64 && d != 128) return LSSAR_ERR_HEADDIM;
    if (dtype != LSSAR_DTYPE_BF16 && dtype != LSSAR_DTYPE_FP16) return LSSAR_ERR_DTYPE;
    if (!k) Hk = 0;
    if (B < 1 || L < 1 || H < 1 || (k && Hk < 1) || L > (1 << 24) || (long long)H + Hk > (1 << 24) ||
        (unsigned long long)B * L > (1ULL << 34) || (unsigned long long)B * L * (H + Hk) > kMaxElems / d)
        return LSSAR_ERR_SHAPE;
    Rope r = {};
    int st = rotary_table(rotary, d, &r.table);
    if (st != LSSAR_OK) return st;
    Range in[2] = {}, out[2] = {};
    if ((st = rope_view(q, qs, q_out, B, H, L, d, &r.v[0], &in[0], &out[0])) != LSSAR_OK) return st;
    if (k && (st = rope_view(k, ks, k_out, B, Hk, L, d, &r.v[1], &in[1], &out[1])) != LSSAR_OK) return st;
    if (misaligned(positions, 4)) return LSSAR_ERR_ALIGN;
    const Range pos = {positions, (size_t)B * (per_token ? L : 1) * 4};
    // each output against everything that is read or written beside its own input
    for (int i = 0; i < (k ? 2 : 1); ++i) {
        const int o = 1 - i;
        if (overlap(out[i], pos)) return LSSAR_ERR_ALIAS;
        if (r.v[i].x != r.v[i].y && overlap(out[i], in[i])) return LSSAR_ERR_ALIAS;
        if (!k) continue;
        for (const Range &x : {in[o], out[o]})
            if (overlap(out[i], x) &&
                !(r.v[i].x == r.v[i].y && x.p == in[o].p && slices_apart(r.v[0].xs, r.v[0].x, H, r.v[1].xs, r.v[1].x, Hk, B, L, d)))
                return LSSAR_ERR_ALIAS;
    }
    r.B = B;
    r.L = L;
    r.d = d;
    r.half = dtype == LSSAR_DTYPE_FP16;
    r.back = back;
    r.positions = positions;
    r.per_token = per_token != 0;
    return launch_rope(r, stream) == cudaSuccess ? LSSAR_OK : LSSAR_ERR_CUDA;
}

}  // namespace

}  // namespace lssar

extern "C" {

int lssar_rope(const void *q, const long long *q_strides, void *q_out, int H, const void *k, const long long *k_strides,
               void *k_out, int Hk, int B, int L, int d, int dtype, const lssar_rotary_t *rotary, const int *positions,
               int per_token, cudaStream_t stream) {
    return lssar::rope_call(q, q_strides, q_out, H, k, k_strides, k_out, Hk, B, L, d, dtype, rotary, positions, per_token, false, stream);
}

int lssar_rope_bwd(const void *q, const long long *q_strides, void *q_out, int H, const void *k, const long long *k_strides,
                   void *k_out, int Hk, int B, int L, int d, int dtype, const lssar_rotary_t *rotary,
                   const int *positions, int per_token, cudaStream_t stream) {
    return lssar::rope_call(q, q_strides, q_out, H, k, k_strides, k_out, Hk, B, L, d, dtype, rotary, positions, per_token, true, stream);
}

}  // extern "C"
