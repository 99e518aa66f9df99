// Paged cache, attention of a chunk: row t < counts[b] of a sequence is row
// i = lens[b] - counts[b] + t + 1 of the attention, in every mode.
//
// One warp per row: a pass over the row's keys for the maximum of the scores z and the sum
// of the normaliser phi, a second for the weights (lanes over keys) and the values (lanes
// over columns).  Everything in fp32 from the inputs' own bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"
#include "row_weights.cuh"
#include "tc_host.cuh"

namespace lssar {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float2 pair_of(uint32_t x, bool half) {
    if (half) return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attend_rows(const __grid_constant__ PagedAttend a, float scale) {
    __shared__ float qs[kWarps][D];
    const PagedCache &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.H / c.Hkv;
    const long long rows = (long long)c.B * a.H * a.n;
#pragma unroll 1
    for (long long r = (long long)blockIdx.x * kWarps + warp; r < rows; r += (long long)gridDim.x * kWarps) {
        const int t = (int)(r % a.n), hq = (int)(r / a.n % a.H), b = (int)(r / a.n / a.H), h = hq / G;
        const int len = c.lens[b], cnt = a.counts ? a.counts[b] : a.n;
        bool bad = len < 0 || len > c.capacity() || cnt < 0 || cnt > a.n || cnt > len;
        if (bad) atomicCAS(c.err, 0u, (unsigned)kErrPagedLength);
        if (!bad && t >= cnt) continue;
        const int *table = c.table + (size_t)b * c.max_pages;
        bool no_page = false;
        for (int i = lane; !bad && i * c.page_size < len; i += 32) no_page |= (unsigned)table[i] >= (unsigned)c.n_pages;
        if (no_page) atomicCAS(c.err, 0u, (unsigned)kErrPagedPage);
        bad |= __any_sync(0xffffffffu, no_page);
        uint16_t *out = static_cast<uint16_t *>(a.out) + (size_t)r * D;
        if (bad) {
            for (int x = lane; x < D; x += 32) out[x] = 0x7fff;   // a NaN in both types
            continue;
        }
        const uint16_t *q = static_cast<const uint16_t *>(a.q) + b * a.qs[0] + hq * a.qs[1] + t * a.qs[2];
        float qq = 0.f;
        __syncwarp();
        for (int x = lane; x < D / 2; x += 32) {
            const float2 v = pair_of(reinterpret_cast<const uint32_t *>(q)[x], c.half);
            qs[warp][2 * x] = v.x;
            qs[warp][2 * x + 1] = v.y;
            qq += v.x * v.x + v.y * v.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) qq += __shfl_xor_sync(0xffffffffu, qq, o);
        __syncwarp();
        const int n = len - cnt + t + 1;
        const bool raw = !uses_normalised_qk(a.mode);
        const float f = raw ? scale : scale * logf((float)n) / fmaxf(sqrtf(qq), 1e-12f);
        auto at = [&](int j) { return table[j / c.page_size] * c.page_stride + ((size_t)h * c.page_size + j % c.page_size) * D; };
        auto score = [&](int j) {
            const uint32_t *k = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(c.k) + at(j));
            float dot = 0.f, kk = 0.f;
#pragma unroll 8
            for (int x = 0; x < D / 2; ++x) {
                const float2 v = pair_of(k[x], c.half);
                dot += qs[warp][2 * x] * v.x + qs[warp][2 * x + 1] * v.y;
                kk += v.x * v.x + v.y * v.y;
            }
            return raw ? dot * f : dot * f / fmaxf(sqrtf(kk), 1e-12f);
        };
        float2 st = make_float2(-3e38f, 0.f);
        for (int j = lane; j < n; j += 32) {
            const float z = score(j), m = fmaxf(st.x, z);
            st.y = raw ? st.y * exp2f(st.x - m) + exp2f(z - m) : st.y + phi(a.mode, z, 0.f);
            st.x = m;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, st.x, o), s2 = __shfl_xor_sync(0xffffffffu, st.y, o), m = fmaxf(st.x, m2);
            st = make_float2(m, raw ? st.y * exp2f(st.x - m) + s2 * exp2f(m2 - m) : st.y + s2);
        }
        const RowConstants rc = row_constants(a.mode, n, st);
        const float lift = exp2f(-fminf(st.x, 0.f));
        float sum = 0.f, acc[D / 32] = {};
        for (int j0 = 0; j0 < n; j0 += 32) {
            float w = 0.f;
            if (j0 + lane < n) {
                const float z = score(j0 + lane);
                w = is_reweight(a.mode) ? powi(above_offset(a.mode, make_float2(z, z), rc), a.p).x
                    : raw               ? exp2f(z - st.x)
                                        : phi(a.mode, z, 0.f) * lift;
            }
            sum += w;
            for (int j = 0; j < min(32, n - j0); ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
                const uint16_t *v = static_cast<const uint16_t *>(c.v) + at(j0 + j);
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    const float2 e = pair_of(reinterpret_cast<const uint32_t *>(v)[x * 32 + lane], c.half);
                    acc[2 * x] += wj * e.x;
                    acc[2 * x + 1] += wj * e.y;
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = 1.f / sum;
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
            reinterpret_cast<uint32_t *>(out)[x * 32 + lane] =
                c.half ? ptx::pack_f16x2(acc[2 * x] * inv, acc[2 * x + 1] * inv) : ptx::pack_bf16x2(acc[2 * x] * inv, acc[2 * x + 1] * inv);
    }
}

}  // namespace

size_t paged_attend_workspace_bytes(const PagedAttend &, int) { return 0; }

cudaError_t launch_paged_attend(const PagedAttend &pr, void *, int sms, cudaStream_t stream) {
    PagedAttend a = pr;
    const cudaError_t e = error_word_ptr(&a.c.err);
    if (e != cudaSuccess) return e;
    const float scale = uses_normalised_qk(a.mode) ? score_qmul(a.c.d) : 1.4426950408889634f / sqrtf((float)a.c.d);
    const long long rows = ((long long)a.c.B * a.H * a.n + kWarps - 1) / kWarps, most = 16LL * sms;
    if (a.c.d == 64) attend_rows<64><<<(unsigned)(rows < most ? rows : most), kWarps * 32, 0, stream>>>(a, scale);
    else attend_rows<128><<<(unsigned)(rows < most ? rows : most), kWarps * 32, 0, stream>>>(a, scale);
    return cudaGetLastError();
}

}  // namespace lssar
