// Paged cache, decode: one new query row per head against a sequence's pages,
// in every mode of the forward (row i = the sequence's length), grouped heads,
// and the attention weight that each cached token receives added up.
//
// One CTA per (sequence, query head): the scores z_j of the row go to a
// scratch row, their maximum and normaliser sum give the row's constants, the
// weights replace the scores and the value rows are summed.  A second kernel
// adds the normalised weights of each key head's group to its tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"
#include "row_weights.cuh"
#include "tc_host.cuh"

namespace lssar {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    return static_cast<float>(x);
}

__device__ float block_reduce(float x, bool is_max, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = is_max ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float r = red[0];
    for (int w = 1; w < kThreads / 32; ++w) r = is_max ? fmaxf(r, red[w]) : r + red[w];
    return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_rows(const PagedDecode a, float *__restrict__ z_all, float *__restrict__ wsum) {
    const PagedCache &c = a.c;
    __shared__ float qs[D], red[kThreads / 32], acc[kThreads / D][D];
    __shared__ int bad;
    const int b = blockIdx.x / a.H, hq = blockIdx.x % a.H, h = hq / (a.H / c.Hkv);
    const int n = paged_len(c, b);
    const bool raw = !uses_normalised_qk(a.mode);
    float *z = z_all + (size_t)blockIdx.x * c.capacity();
    T *out = static_cast<T *>(a.out) + (size_t)blockIdx.x * D;
    float ss = 0.f;
    if (threadIdx.x == 0) bad = c.lens[b] != n;
    for (int t = threadIdx.x; t < D; t += kThreads) {
        qs[t] = to_f32(static_cast<const T *>(a.q)[b * a.q_b + hq * a.q_h + t]);
        ss += qs[t] * qs[t];
    }
    ss = block_reduce(ss, false, red);
    const float log2e = 1.4426950408889634f;
    const float scale = raw ? log2e * rsqrtf((float)D)
                            : log2e * logf((float)D) * logf((float)max(n, 1)) / fmaxf(sqrtf(ss), 1e-12f);
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int j = threadIdx.x >> 5; j < n; j += kThreads / 32) {
        const int pg = paged_page(c, b, j / c.page_size);
        float dot = 0.f, kss = 0.f;
        if (pg < 0) {
            bad = 1;
        } else {
            const T *k = static_cast<const T *>(c.k) + pg * c.page_stride + ((size_t)h * c.page_size + j % c.page_size) * D;
            for (int t = lane; t < D; t += 32) {
                const float x = to_f32(k[t]);
                dot += x * qs[t];
                kss += x * x;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
            kss += __shfl_xor_sync(0xffffffffu, kss, o);
        }
        const float zj = raw ? scale * dot : scale * dot * rsqrtf(fmaxf(kss, 1e-24f));
        if (lane == 0) z[j] = zj;
        m = fmaxf(m, zj);
    }
    m = block_reduce(m, true, red);   // its barriers also publish the scores
    float s1 = 0.f;
    for (int j = threadIdx.x; j < n; j += kThreads) s1 += phi(a.mode, z[j], m);
    s1 = block_reduce(s1, false, red);
    float kappa = 1.f, beta = 0.f;
    if (is_reweight(a.mode)) {
        const float theta = n <= 3 ? 0.f : s1 / (float)n, top = phi(a.mode, m, m), den = top - theta;
        const bool uniform = !(den > 1e-5f * top + 2e-5f);
        kappa = uniform ? 0.f : 1.f / den;
        beta = uniform ? 1.f : -theta * kappa;
    }
    float w2 = 0.f;
    for (int j = threadIdx.x; j < n; j += kThreads) {
        float w = fmaf(phi(a.mode, z[j], m), kappa, beta);
        if (is_reweight(a.mode)) w = powi(fmaxf(w, 0.f), a.p);
        z[j] = w;
        w2 += w;
    }
    w2 = block_reduce(w2, false, red);   // its barriers also publish the weights
    const int col = threadIdx.x % D;
    float o = 0.f;
    for (int j = threadIdx.x / D; j < n; j += kThreads / D) {
        const int pg = paged_page(c, b, j / c.page_size);
        if (pg >= 0)
            o += z[j] * to_f32(static_cast<const T *>(c.v)[pg * c.page_stride + ((size_t)h * c.page_size + j % c.page_size) * D + col]);
    }
    acc[threadIdx.x / D][col] = o;
    __syncthreads();
    if (threadIdx.x < D) {
        o = 0.f;
        for (int g = 0; g < kThreads / D; ++g) o += acc[g][threadIdx.x];
        out[threadIdx.x] = T(bad ? NAN : n == 0 ? 0.f : o / w2);
    }
    if (threadIdx.x == 0) wsum[blockIdx.x] = bad ? NAN : w2;
}

__global__ void __launch_bounds__(kThreads) paged_scores(const PagedDecode a, const float *__restrict__ w, const float *__restrict__ wsum) {
    const PagedCache &c = a.c;
    const int cap = c.capacity(), G = a.H / c.Hkv;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)c.B * c.Hkv * cap) return;
    const int bh = (int)(i / cap), b = bh / c.Hkv, slot = (int)(i % cap);
    if (slot >= paged_len(c, b)) return;
    float s = 0.f;
    for (int g = 0; g < G; ++g) {
        const int row = b * a.H + (bh % c.Hkv) * G + g;
        s += w[(size_t)row * cap + slot] / wsum[row];
    }
    a.scores_out[i] = a.scores[i] + s;
}

}  // namespace

size_t paged_decode_workspace_bytes(const PagedDecode &pr, int) {
    return ((size_t)pr.c.B * pr.H * pr.c.capacity() + (size_t)pr.c.B * pr.H) * 4;
}

cudaError_t launch_paged_decode(const PagedDecode &pr, void *ws, int, cudaStream_t stream) {
    PagedDecode a = pr;
    cudaError_t e = error_word_ptr(&a.c.err);
    if (e != cudaSuccess) return e;
    const int rows = a.c.B * a.H;
    float *z = static_cast<float *>(ws), *wsum = z + (size_t)rows * a.c.capacity();
    if (a.c.half)
        (a.c.d == 64 ? paged_rows<__half, 64> : paged_rows<__half, 128>)<<<rows, kThreads, 0, stream>>>(a, z, wsum);
    else
        (a.c.d == 64 ? paged_rows<__nv_bfloat16, 64> : paged_rows<__nv_bfloat16, 128>)<<<rows, kThreads, 0, stream>>>(a, z, wsum);
    if (a.scores) {
        const long long slots = (long long)a.c.B * a.c.Hkv * a.c.capacity();
        paged_scores<<<(unsigned)((slots + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a, z, wsum);
    }
    return cudaGetLastError();
}

}  // namespace lssar
