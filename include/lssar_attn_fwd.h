/*
 * lssar_attn_fwd.h -- C ABI of the GB300 (sm_103a) causal LSSAR attention forward.
 *
 * The operation is the attention forward defined in the papernotes.org notes on
 * "Softplus Attention with Re-weighting Boosts Length Extrapolation in Large
 * Language Models" (arXiv 2501.13428):
 *
 *   Key design 1 (LSSA): q_i <- q_i/||q_i||_2, k_j <- k_j/||k_j||_2,
 *       A_ij = Softplus(ln d * ln i * q_i.k_j) for j <= i (0 above the diagonal,
 *       a multiplicative mask applied after the Softplus), then each row of A is
 *       divided by its sum.  i is the 1-based row index (tokens attended).
 *   Key design 2 (re-weighting): A_ij <- max(i*A_ij - O_i, 0)^p with O_i = 0 for
 *       rows 1..3 and 1 otherwise, then each row is divided by its sum again.
 *   The output row i is sum_j A_ij v_j.
 *   Background (softmax mode): A = Softmax(q.k^T / sqrt(d) + causal -inf mask).
 *   Ablation table (modes 3, 4): re-weighting applied to the softmax attention
 *       above, and to LSSA with Sigmoid(x) = 1/(1+e^-x) in place of Softplus.
 *
 * A re-weighted row whose entries are all zero (possible only when the LSSA
 * row is exactly uniform) is 0/0 in the notes; this library returns the
 * uniform prefix mean for it.  Norms are clamped at 1e-12.
 *
 * Conventions shared by every entry point:
 *   - q, k, v, out are DEVICE pointers to bfloat16 tensors of shape
 *     [B, H, L, d], contiguous (d fastest), each 16-byte aligned.  The caller
 *     owns them; out must not overlap q, k or v.
 *   - Calls are asynchronous on `stream` (0 = legacy default stream) and return
 *     once the work is enqueued.  Errors in the arguments are reported before
 *     anything is launched; nothing is written to `out` in that case.
 *   - Temporary device memory is taken stream-ordered from a memory pool owned
 *     by the library and released stream-ordered on the same stream.
 *   - Thread-safe: no mutable global state besides the lazily created pool
 *     (guarded) and the device error word (see lssar_device_error_word).
 *   - The device addresses of the library's own device variables (the error
 *     word, the fixed scratch of lssar_attn_fwd_noalloc) and its memory pool
 *     are looked up once per device and kept: after cudaDeviceReset (or any
 *     other teardown of a device's primary context) the library must not be
 *     used on that device again in the same process.
 */
#ifndef LSSAR_ATTN_FWD_H
#define LSSAR_ATTN_FWD_H

#ifdef __cplusplus
extern "C" {
#endif

/* Same types as the CUDA runtime's cudaStream_t and cudaEvent_t. */
typedef struct CUstream_st *cudaStream_t;
typedef struct CUevent_st *cudaEvent_t;

typedef enum {
    LSSAR_MODE_SOFTMAX = 0,    /* Softmax(q.k^T/sqrt(d)) on raw q, k (Background)    */
    LSSAR_MODE_LSSA = 1,       /* Key design 1 only                                   */
    LSSAR_MODE_LSSAR = 2,      /* Key design 1 followed by Key design 2               */
    LSSAR_MODE_SOFTMAX_RW = 3, /* ablation: Softmax(q.k^T/sqrt(d)), then Key design 2 */
    LSSAR_MODE_SIGMOID_RW = 4  /* ablation: Key design 1 with Sigmoid in place of
                                  Softplus, then Key design 2                         */
} lssar_mode_t;

typedef enum {
    LSSAR_OK = 0,
    LSSAR_ERR_NULL = -1,    /* a tensor pointer is NULL                               */
    LSSAR_ERR_SHAPE = -2,   /* B, H or L < 1, L > 2^24, or B*H*L*d beyond 2^40         */
    LSSAR_ERR_HEADDIM = -3, /* d is not 64 or 128                                     */
    LSSAR_ERR_P = -4,       /* re-weighting mode (2, 3, 4) with p < 1 or p > 1024     */
    LSSAR_ERR_MODE = -5,    /* unknown mode                                           */
    LSSAR_ERR_ALIGN = -6,   /* a pointer is not 16-byte aligned                       */
    LSSAR_ERR_CUDA = -7,    /* a CUDA call failed (launch, pool allocation, ...)      */
    LSSAR_ERR_ALIAS = -8,   /* an output overlaps an input (or another output)         */
    LSSAR_ERR_SCRATCH = -9, /* lssar_attn_fwd_noalloc: problem needs more scratch than
                               LSSAR_NOALLOC_SCRATCH_BYTES                            */
    LSSAR_ERR_PAGE = -10,   /* paged cache: page_size not a multiple of 8 in 8..256, no
                               page, or a page_stride that does not fit               */
    LSSAR_ERR_DTYPE = -11,  /* paged cache: dtype is not an lssar_dtype_t              */
    LSSAR_ERR_KEEP = -12,   /* lssar_paged_evict: keep < 1, recent < 0, sinks < 0 or
                               recent + sinks > keep                                  */
    LSSAR_ERR_ROTARY = -13  /* rotary positions: a field of lssar_rotary_t out of range */
} lssar_status_t;

/*
 * Causal attention forward, computed by the tensor-core (tcgen05/TMEM/TMA)
 * kernel for sm_103a.
 *   q, k, v : [B, H, L, d] bfloat16, device, read only.
 *   out     : [B, H, L, d] bfloat16, device, written (row i of head (b, h)).
 *   p       : integer exponent of the re-weighting (modes 2, 3, 4: 1..1024;
 *             ignored in modes 0, 1).
 *   mode    : lssar_mode_t.
 * Returns LSSAR_OK or a negative lssar_status_t.
 * Numerics of LSSAR mode with p >= 4: the weight pass evaluates the softplus
 * of a row as z + 2^-|z| / ln 2 (one exponential, z = log2(e) x) instead of
 * log2(1 + 2^z) when a bound computed from the row's statistics (its
 * threshold, spread, length and p) guarantees that the row's weights change
 * in sum by at most 2e-4 of their total (the output by at most 4e-4 max|v|);
 * other rows keep log2(1 + 2^z).  Setting LSSAR_EXACT_WEIGHTS=1 in the
 * environment keeps every row on log2(1 + 2^z) (read at each call).
 */
int lssar_attn_fwd(const void *q, const void *k, const void *v, void *out,
                   int B, int H, int L, int d, int p, int mode, cudaStream_t stream);

/*
 * lssar_attn_fwd with one re-weighting exponent per head: head h (of every
 * batch entry) uses p_per_head[h].  The notes leave an adaptive or learnable p
 * open (Limitations: p = 15 is empirical; Key findings: the best sparsity
 * depends on the length); a per-head p is what such a model needs at
 * inference time.
 *   p_per_head : HOST array of H ints, each in 1..1024, read before return.
 *   mode       : a re-weighting mode (2, 3 or 4); other modes return
 *                LSSAR_ERR_P.  H must be at most 256 (LSSAR_ERR_P otherwise).
 * Other arguments, results and errors as lssar_attn_fwd.
 */
int lssar_attn_fwd_heads_p(const void *q, const void *k, const void *v, void *out,
                           int B, int H, int L, int d, const int *p_per_head, int mode,
                           cudaStream_t stream);

/*
 * Training forward: lssar_attn_fwd that also saves, per query row, what the
 * backward pass needs (the notes train GPT-2 models with this attention).
 *   stats : [B, H, L, 4] float32, device, 16-byte aligned, written:
 *           {m, kappa, beta, W} per row, in the kernel's log2 units
 *           (z = log2(e) * x):  phi(z) = log2(1 + 2^z) (LSSA/LSSAR),
 *           2^(z - m) (softmax normalisers), 1/(1 + 2^-z) (sigmoid); the row's
 *           weights are w = max(phi kappa + beta, 0)^p with W = sum_j w
 *           (kappa = 1, beta = 0, p = 1 without re-weighting).  A row read as
 *           the uniform prefix mean has kappa = 0, beta = 1, W = i.
 * Must not overlap q, k, v or out.  Other arguments, results and errors as
 * lssar_attn_fwd (LSSAR_ERR_NULL for a NULL stats, LSSAR_ERR_ALIGN, ALIAS).
 */
int lssar_attn_fwd_train(const void *q, const void *k, const void *v, void *out, float *stats,
                         int B, int H, int L, int d, int p, int mode, cudaStream_t stream);

/*
 * Backward pass on the tensor cores: gradients of sum(dout * out) with
 * respect to q, k and v, from the row statistics of lssar_attn_fwd_train.
 * Same operation, arguments, results and errors as lssar_attn_bwd_simt below.
 * Two persistent tcgen05 kernels: a pass over each 128-query tile (dq, and the
 * per-query terms D_i = dout_i . out_i and the re-weighting threshold's
 * gradient) and a pass over each 128-key tile (dk, dv), each applying the
 * gradient of the L2 row normalisation to its own tile before it writes;
 * scores use fp16 normalised rows as in the forward, the gradient products
 * fp16 (normalised modes) or bf16 (softmax modes) with fp32 accumulation.
 * Scratch: 256 + round_up(4*B*H, 256) + 2*round_up(2*B*H*L*d, 256)
 * (normalised modes only) + round_up(32*B*H*ceil(L/128)*128, 256) bytes from
 * the library's stream-ordered pool.
 */
int lssar_attn_bwd(const void *q, const void *k, const void *v, const void *dout,
                   const float *stats, void *dq, void *dk, void *dv,
                   int B, int H, int L, int d, int p, int mode, cudaStream_t stream);

/*
 * Training with one re-weighting exponent per head (the notes leave an
 * adaptive or learnable p open: Limitations; training is where such a p would
 * be chosen).  lssar_attn_fwd_train_heads_p is lssar_attn_fwd_train, and
 * lssar_attn_bwd_heads_p is lssar_attn_bwd, with head h (of every batch entry)
 * using p_per_head[h]; pass the same array to both.
 *   p_per_head : HOST array of H ints, each in 1..1024, read before return.
 *   mode       : a re-weighting mode (2, 3 or 4); other modes return
 *                LSSAR_ERR_P.  H must be at most 256 (LSSAR_ERR_P otherwise).
 * Other arguments, results and errors as lssar_attn_fwd_train / lssar_attn_bwd.
 */
int lssar_attn_fwd_train_heads_p(const void *q, const void *k, const void *v, void *out, float *stats,
                                 int B, int H, int L, int d, const int *p_per_head, int mode,
                                 cudaStream_t stream);
int lssar_attn_bwd_heads_p(const void *q, const void *k, const void *v, const void *dout,
                           const float *stats, void *dq, void *dk, void *dv,
                           int B, int H, int L, int d, const int *p_per_head, int mode,
                           cudaStream_t stream);

/*
 * Backward pass: gradients of sum(dout * out) with respect to q, k and v,
 * given the row statistics of the forward (lssar_attn_fwd_train with the same
 * q, k, v, B, H, L, d, p, mode).  Chain rule through the steps of Key designs
 * 1-2: the derivative of the L1 normalisations, of the re-weighting threshold
 * (its row sum S1), of softplus / sigmoid / exp and of the L2 row
 * normalisation; a uniform row passes no gradient to its scores.  The
 * forward's output is not needed: dout_i . out_i is formed from the
 * recomputed weights, free of the output's bf16 rounding.
 *   q, k, v, dout : [B, H, L, d] bfloat16, device, read only.
 *   stats         : [B, H, L, 4] float32 from lssar_attn_fwd_train.
 *   dq, dk, dv    : [B, H, L, d] bfloat16, device, written; they must not
 *                   overlap each other or any input (LSSAR_ERR_ALIAS).
 * Scratch (8*B*H*L bytes) comes from the library's stream-ordered pool.  Other
 * arguments and errors as lssar_attn_fwd.
 *
 * This entry point runs a plain CUDA-core implementation (one warp per query
 * row for dq, one warp per key row for dk and dv, fp32, libm
 * transcendentals); it is the cross-check for the tensor-core backward.
 */
int lssar_attn_bwd_simt(const void *q, const void *k, const void *v, const void *dout,
                        const float *stats, void *dq, void *dk, void *dv,
                        int B, int H, int L, int d, int p, int mode, cudaStream_t stream);

/*
 * Decode step: the forward for ONE new query row per head, at position L
 * (1-based, i.e. it attends to all L cached tokens, itself included), for
 * every mode above.  Equal to row L of lssar_attn_fwd on the full sequence
 * (the notes evaluate a model trained at 1K tokens at 2K-8K: this is that
 * inference step).
 *   q       : [B, H, d] bfloat16, device (the new token's query).
 *   k_cache : [B, H, L, d] bfloat16, device (keys 1..L, the new one last).
 *   v_cache : [B, H, L, d] bfloat16, device.
 *   out     : [B, H, d] bfloat16, device, written.
 * Bound by HBM: K and V are read once.  Each head's cache is cut into up to
 * 16 chunks of at most 4096 keys that form one thread-block cluster: the
 * chunks' statistics and partial outputs meet in distributed shared memory
 * and the scores stay in shared memory, so a step is one launch that touches
 * no other global memory.  Longer caches (over 65536 keys per head) take a
 * cooperative launch with a grid barrier, or three launches when that grid
 * cannot be resident at once; those paths keep scores and partials in a
 * float scratch of about 4*B*H*L bytes from the library's pool.  The
 * environment variable LSSAR_DECODE_PATH=grid (or split) makes a call skip
 * the cluster path (or use the three launches), to test those paths at small
 * sizes.  Same errors as lssar_attn_fwd.
 */
int lssar_attn_decode(const void *q, const void *k_cache, const void *v_cache, void *out,
                      int B, int H, int L, int d, int p, int mode, cudaStream_t stream);

/*
 * Paged key-value cache: the decode step for sequences of different lengths
 * whose keys and values lie in pages, with grouped heads (query head h reads
 * key head h / (H / Hkv)).
 *
 *   k_pages, v_pages : 16-bit elements (dtype), device, 16-byte aligned.  Row r
 *       of page g and key head h starts at element
 *       g * page_stride + (h * page_size + r) * d: [n_pages, Hkv, page_size, d],
 *       whose first stride may be larger than a page (both share it), so that K
 *       and V can be slices of one buffer.
 *   table : [B, max_pages] int32, device.  Slot s of sequence b lies in page
 *       table[b][s / page_size], row s % page_size.  Entries past the last page
 *       in use are not read.
 *   lens  : [B] int32, device: the tokens cached for each sequence, 0 ..
 *       max_pages * page_size (the capacity).
 *
 * The contents of table and lens are on the device, so that the kernels check
 * them: a length outside 0..capacity records code 51 in the device error word,
 * a page number outside 0..n_pages-1 code 52, and no access is made through
 * either; what each call then does is said below.  Sequences may share pages
 * that are only read.
 */
typedef enum { LSSAR_DTYPE_BF16 = 0, LSSAR_DTYPE_FP16 = 1 } lssar_dtype_t;

typedef struct {
    void *k_pages;
    void *v_pages;
    const int *table;
    const int *lens;
    long long page_stride;   /* elements from one page to the next, a multiple of 8 */
    int n_pages;
    int max_pages;           /* columns of table; max_pages * page_size <= 2^24 */
    int page_size;           /* tokens per page: a multiple of 8 in 8..256 */
    int B, Hkv, d;           /* d is 64 or 128 */
    int dtype;               /* lssar_dtype_t */
} lssar_paged_cache_t;

/*
 * Append: token t < counts[b] of sequence b goes to slot lens[b] + t.
 *   k_new, v_new : [B, Hkv, n, d] of the cache's type, device; k_strides and
 *       v_strides are HOST arrays of the element strides of (B, Hkv, n), each a
 *       multiple of 8 where its dimension is above 1 (slices of a fused
 *       projection need no copy).  Rows t >= counts[b] are not read.
 *   n      : 0 .. 2^24 (0: k_new and v_new may be NULL).
 *   counts : [B] int32, device, 0..n each; NULL: n for every sequence.
 *   first_positions : [B] int32, device: position of token 0; NULL: lens[b].
 *   scores : [B, Hkv, capacity] float32, or NULL: the new slots become 0.
 *   positions : [B, Hkv, capacity] int32, or NULL: the new slots become
 *       first_positions[b] + t.
 *   lens_out : [B] int32, written: lens[b] + counts[b].  Not lens itself.
 * Nothing else is written.  Two sequences must not append to one page.  A
 * sequence with a bad length or count, or whose new length passes the
 * capacity, is left alone (code 51, lens_out[b] = lens[b]); rows of a bad page
 * number are dropped (code 52).
 * Errors: LSSAR_ERR_NULL, SHAPE, HEADDIM, PAGE, DTYPE, ALIGN (a pointer or a
 * stride), ALIAS (an output overlaps anything else; k_new, v_new, counts or
 * first_positions overlap the pages), CUDA.
 */
int lssar_paged_append(const lssar_paged_cache_t *cache, const void *k_new, const long long *k_strides,
                       const void *v_new, const long long *v_strides, int n, const int *counts,
                       const int *first_positions, float *scores, int *positions, int *lens_out, cudaStream_t stream);

/*
 * Decode: row i = lens[b] of the attention in every mode, for one new query
 * per head against the sequence's cached tokens, the new one among them
 * (append first).  i is the number of cached tokens, also after an eviction.
 *   q   : [B, H, d] of the cache's type; q_strides is a HOST array of the
 *         element strides of (B, H), multiples of 8 where the dimension is above 1.
 *   out : [B, H, d] contiguous, of the cache's type, written.
 *   H   : query heads, a multiple of Hkv, at most 128 * Hkv.
 *   scores, scores_out : [B, Hkv, capacity] float32, both or neither:
 *         scores_out[b][h][s] = scores[b][h][s] + the normalised weights of slot
 *         s of the query heads of h, for s < lens[b]; other slots are not
 *         written.  scores_out may be scores itself.
 * A sequence of length 0 gets out = 0.  One with a bad length gets NaN rows and
 * no scores; with a bad page number, NaN rows and NaN scores in the heads.
 * The sums have a fixed order: the same call on the same device gives the same
 * bits.  Two launches (softmax, LSSA) or three (re-weighting modes, which need a
 * row's scores before its weights).  K and V are read once for each of the
 * n8 = ceil(H / (8 Hkv)) blocks of query heads of a key head.  Scratch from the
 * library's pool, with h8 = min(H / Hkv, 8) heads for every block (groups that
 * are no multiple of 8 leave some unused): 4 * (d + 4) bytes for each of
 * (B * Hkv * n8 + 3 * SMs) * h8 partial sums at most, and in the re-weighting
 * modes or with scores 4 bytes for each of B * Hkv * n8 * h8 heads and slot that
 * the table has room for (rounded up to a multiple of 8192 / d), whatever the
 * lengths.  Errors as lssar_paged_append, and LSSAR_ERR_MODE, LSSAR_ERR_P; LSSAR_ERR_SHAPE also when B * Hkv * ceil(H / (8 Hkv)) *
 * ceil(capacity / 64) passes 2^31 - 2^16.
 */
int lssar_paged_decode(const lssar_paged_cache_t *cache, const void *q, const long long *q_strides, void *out, int H,
                       int p, int mode, const float *scores, float *scores_out, cudaStream_t stream);

/*
 * Evict: of each (sequence, key head) with n = lens[b] > keep, the `keep`
 * tokens of the highest rank stay.  Rank: protected tokens first (position <
 * sinks, or position > newest - recent, newest being the largest position of
 * the row), then by score, equal scores (-0 = 0) by the lower slot, NaN last.
 * Kept tokens in slots >= keep move into the slots < keep that were evicted,
 * the j-th into the j-th in the order of the slots; the others stay where they
 * are.  Keys, values, scores and positions move; a row of K and V at or behind
 * slot `keep` is left as it was.
 *   scores, positions : [B, Hkv, capacity], as the two calls above fill them.
 *   scores_out, positions_out : the slots below the new length are written; both
 *         may be the inputs themselves (then only the moved slots are written),
 *         otherwise they must overlap nothing.
 *   lens_out : [B] int32, written: min(lens[b], keep).  Not lens itself.
 * Sequences must not share pages with one another here, except pages in which
 * nothing moves.  A bad length: nothing moves, lens_out[b] = lens[b]; rows
 * to or from a bad page number are not copied.
 * Two launches: the selection, a thread-block cluster per (sequence, key head),
 * and the moves.  Scratch: B * Hkv * (8 keep + 4) bytes.  Errors as above, and
 * LSSAR_ERR_KEEP.
 */
int lssar_paged_evict(const lssar_paged_cache_t *cache, const float *scores, const int *positions, int keep, int recent,
                      int sinks, float *scores_out, int *positions_out, int *lens_out, cudaStream_t stream);

/*
 * Attention of a chunk: the last counts[b] rows of the attention over the
 * lens[b] cached tokens of each sequence, in every mode (a prompt in pieces, or
 * whole; single tokens beside chunks).  Row t < counts[b] is row
 * i = lens[b] - counts[b] + t + 1: it attends to the slots 0..i-1, its own the
 * last of them (append first).  i counts cached tokens, also after an eviction.
 *   q   : [B, H, n, d] of the cache's type; q_strides is a HOST array of the
 *         element strides of (B, H, n), multiples of 8 where the dimension is
 *         above 1.  Rows t >= counts[b] are not read.
 *   n   : rows per sequence, 1..2^24; H: query heads, a multiple of Hkv, at most
 *         128 * Hkv.
 *   counts : [B] int32, device, 0..min(n, lens[b]) each; NULL: n for every sequence.
 *   out : [B, H, n, d] contiguous, of the cache's type.  Rows t >= counts[b] are
 *         not written.
 * A bad length or count (code 51) gives NaN in all n rows of that sequence, a bad
 * page number among the pages in use (code 52) in the rows that attend to one of
 * that page's slots.  What the rows of pages past lens[b] hold does not matter.
 * A value that is infinite or NaN among the cached tokens reaches the rows of
 * the chunk that attend to it, and may reach rows up to 383 slots before it.
 * The rows' weights are added up nowhere: an eviction goes by those of
 * lssar_paged_decode.
 * LSSAR weights with p >= 4 as in lssar_attn_fwd: by one exponential where its
 * bound allows, none with LSSAR_EXACT_WEIGHTS=1 in the environment.
 * The sums have a fixed order: the same call on the same device gives the same
 * bits.  Three launches (softmax, LSSA) or four (re-weighting modes).  K and V are
 * read once for each block of T = floor(256 Hkv / H) tokens, K twice in the
 * re-weighting modes and once more for its norms where the mode has them (of every
 * cached token, also of sequences without rows).  Scratch
 * from the library's pool, by what the table and n have room for: 16 bytes for each
 * of B ceil(n / T) blocks; 4 bytes for each key head and slot (modes with norms); 8
 * bytes for each of min(n, T) H / Hkv rows of B Hkv ceil(n / T) + SMs items
 * (re-weighting modes); 8 (d + 2) bytes for each of SMs * min(n, T) H / Hkv rows.
 * Errors as lssar_paged_decode; SHAPE also where
 * B Hkv ceil(n / T) (ceil(capacity / 64) + 7) passes 2^31 - 2^16.
 */
int lssar_paged_attend(const lssar_paged_cache_t *cache, const void *q, const long long *q_strides, void *out, int H,
                       int n, const int *counts, int p, int mode, cudaStream_t stream);

/*
 * Rotary positions (the notes' models are GPT-2 with RoPE): the pair c of a row
 * at position m turns by m * f_c radians, (u, v) -> (u cos - v sin, u sin + v cos),
 *   f_c = base^(-2c / rot_dim), c = 0 .. rot_dim / 2 - 1, before scaling.
 * The pairs are the elements (c, c + rot_dim / 2), or (2c, 2c + 1) where
 * interleaved; elements from rot_dim on are copied.  For contexts longer than
 * the trained one f_c is scaled:
 *   LINEAR  f_c / factor
 *   BASE    base * factor^(rot_dim / (rot_dim - 2)) in place of base
 *   BANDS   f_c (g + (1 - g) / factor), g = clamp((r - low) / (high - low), 0, 1),
 *           r = original_length f_c / (2 pi): pairs that turn often within the
 *           trained length keep their frequency
 * Angles are taken modulo a turn in 64-bit fixed point.  They are off by at most
 * |m| 2^-50 turns (the frequencies' rounding as doubles: 2^-30 at a position of 10^6,
 * 2^-19 at 2^31; with a base of 10000 about 2^-24 there; BANDS: 2 high /
 * (high - low) times as much) and 2^-25 turns (their conversion to fp32).  The products are in
 * fp32, rounded once.
 */
typedef enum {
    LSSAR_ROPE_PLAIN = 0, LSSAR_ROPE_LINEAR = 1, LSSAR_ROPE_BASE = 2, LSSAR_ROPE_BANDS = 3
} lssar_rope_scaling_t;

typedef struct {
    double base;             /* > 1, finite */
    double factor;           /* >= 1, finite (not PLAIN) */
    double low, high;        /* 0 <= low < high, finite (BANDS) */
    int original_length;     /* >= 1 (BANDS) */
    int rot_dim;             /* a multiple of 16 in 16..d */
    int interleaved;         /* 0 or 1 */
    int scaling;             /* lssar_rope_scaling_t */
} lssar_rotary_t;

/*
 * Turns q [B, H, L, d] and k [B, Hk, L, d] (k NULL: q alone) by their positions.
 *   q_strides, k_strides : HOST arrays of the element strides of (B, H, L),
 *         multiples of 8 where the dimension is above 1.
 *   positions : device int32, or NULL: token t is at position t.  per_token 0:
 *         [B], token t of sequence b at positions[b] + t; 1: [B, L].
 *   q_out, k_out : contiguous, apart from everything else; or the input itself
 *         (the same address), which is then turned in place at its own strides (rows
 *         that do not overlap; q and k may be slices of one [B, L, heads, d] buffer).
 * d is 64 or 128, dtype an lssar_dtype_t, H and Hk at least 1.
 * lssar_rope_bwd turns back: the gradients with respect to the inputs from
 * those with respect to the outputs (the same arguments).
 * Errors: LSSAR_ERR_NULL, SHAPE, HEADDIM, DTYPE, ROTARY, ALIGN, ALIAS, CUDA.
 */
int lssar_rope(const void *q, const long long *q_strides, void *q_out, int H, const void *k, const long long *k_strides,
               void *k_out, int Hk, int B, int L, int d, int dtype, const lssar_rotary_t *rotary, const int *positions,
               int per_token, cudaStream_t stream);
int lssar_rope_bwd(const void *q, const long long *q_strides, void *q_out, int H, const void *k, const long long *k_strides,
                   void *k_out, int Hk, int B, int L, int d, int dtype, const lssar_rotary_t *rotary,
                   const int *positions, int per_token, cudaStream_t stream);

/*
 * lssar_paged_append with rotary positions, in one launch: token t < counts[b]
 * of sequence b is at position first_positions[b] + t (NULL: lens[b] + t); its
 * key is turned on its way to the pages, its query turned into q_out.
 *   q : [B, H, n, d] of the cache's type, q_strides as above; H >= 1.
 *   q_out : [B, H, n, d] contiguous, or q itself (in place).  Rows t >= counts[b]
 *         are not written, nor those of a sequence that is left alone; without
 *         counts, apart from q, the latter are zeros.
 * Other arguments, results and errors as lssar_paged_append and lssar_rope.
 */
int lssar_paged_append_rope(const lssar_paged_cache_t *cache, const void *q, const long long *q_strides, void *q_out,
                            int H, const void *k_new, const long long *k_strides, const void *v_new,
                            const long long *v_strides, int n, const lssar_rotary_t *rotary, const int *counts,
                            const int *first_positions, float *scores, int *positions, int *lens_out,
                            cudaStream_t stream);

/*
 * Reserve: page numbers from a list of free pages for counts[b] more tokens of
 * each sequence, so that an append of them fits.  Sequence b holds
 * ceil(lens[b] / page_size) pages; what it needs more comes from the end of the
 * list, in the order of the sequences, and goes to the next columns of its row
 * of table.
 *   table : [B, max_pages] int32, device; only those entries are written.
 *   counts : [B] int32, device, >= 0; NULL: 1 for every sequence.
 *   free_pages : [n_pages] int32, device, read; its first free_count[0] entries
 *         are free pages (free_count: [1] int32, device).
 *   counts_out : [B] int32, written: counts[b] where the sequence has its pages,
 *         0 where it does not: those that need pages, from the first one on whose
 *         needs, added to those before it, pass free_count[0] (they get none).
 *   free_out : [1] int32, written: the free pages left.
 * A bad length or count, or a new length past the capacity, is not served and
 * needs nothing; a free_count outside 0..n_pages serves none (free_out =
 * free_count): code 51.  An entry of the list that is no page of 0..n_pages-1
 * becomes -1 in the table: code 52.
 * page_size as in a cache; B, max_pages, n_pages >= 1, max_pages * page_size <=
 * 2^24.  Outputs overlap nothing else (table is one).
 */
int lssar_paged_reserve(int *table, int max_pages, int page_size, const int *lens, const int *counts, int B,
                        const int *free_pages, int n_pages, const int *free_count, int *counts_out, int *free_out,
                        cudaStream_t stream);

/*
 * Release: the pages of sequence b past its first ceil(lens_new[b] / page_size),
 * up to ceil(lens[b] / page_size), go to the end of the list of free pages, in
 * the order of the sequences and of their tables (after an eviction, or with
 * lens_new[b] = 0 at a sequence's end).  The table stays as it is: entries past
 * a length are not read.
 *   free_pages : [n_pages], written from entry free_count[0] on.
 *   free_out : [1] int32, written: the free pages there are now.
 * A length outside 0..capacity, or a lens_new[b] outside 0..lens[b], releases
 * nothing: code 51.  A free_count outside 0..n_pages, or one that the released
 * pages carry past n_pages: nothing is done, free_out = free_count, code 51.
 * An entry of the table that is no page is passed on as it is, code 52.
 * Pages that sequences share must be released by one of them alone.
 * Sizes and errors as lssar_paged_reserve.
 */
int lssar_paged_release(const int *table, int max_pages, int page_size, const int *lens, const int *lens_new, int B,
                        int *free_pages, int n_pages, const int *free_count, int *free_out, cudaStream_t stream);

/*
 * Same operation and contract as lssar_attn_fwd, computed by a plain CUDA-core
 * kernel (one warp per query row, fp32 throughout, accurate libm softplus).
 * It is a second, independent GPU implementation kept for cross-checking the
 * tensor-core kernel; it is not tuned for speed.
 */
int lssar_attn_fwd_simt(const void *q, const void *k, const void *v, void *out,
                        int B, int H, int L, int d, int p, int mode, cudaStream_t stream);

/*
 * lssar_attn_fwd with timing hooks: records `ev_start` on `stream` before the
 * first kernel of the call (the normalisation prologue, LSSA/LSSAR modes),
 * `ev_main` just before the attention kernel and `ev_end` after it.  Any event
 * may be NULL (not recorded).  Events are created and owned by the caller.
 * Used by the benchmark to time the attention kernel alone; the computation
 * is identical to lssar_attn_fwd.  A non-NULL ev_main costs time: the
 * attention kernel is launched as a programmatic dependent of the prologue
 * (its launch and setup overlap the prologue's tail), and an event recorded
 * between the two makes it wait for the prologue to finish first (about 5 us
 * per call on GB300).
 */
int lssar_attn_fwd_profiled(const void *q, const void *k, const void *v, void *out,
                            int B, int H, int L, int d, int p, int mode, cudaStream_t stream,
                            cudaEvent_t ev_start, cudaEvent_t ev_main, cudaEvent_t ev_end);

/*
 * Size of the fixed device scratch array used by lssar_attn_fwd_noalloc
 * (32 MiB).  Every GPU on which the library is loaded holds it until the
 * process exits.
 */
#define LSSAR_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * lssar_attn_fwd without any device memory allocation.
 *
 * The notes on the method have no counterpart of this: it exists for callers
 * that cannot let a library allocate device memory while it runs -- for
 * example inference-runtime plugins whose execute/enqueue step is not allowed
 * to allocate, hosts that reserve their whole memory budget up front, and
 * latency-critical loops where an allocation could block on the driver.
 *
 * Same operation, arguments and results as lssar_attn_fwd.  The caller still
 * provides q, k, v and out; the temporary data (a work counter and the
 * normalised q and k in fp16: 256 + 2*round_up(2*B*H*L*d, 256) bytes in
 * LSSA/LSSAR mode, 256 bytes in softmax mode) lives in one fixed device array of
 * LSSAR_NOALLOC_SCRATCH_BYTES compiled into the library.  Problems that need
 * more return LSSAR_ERR_SCRATCH before anything is launched (for example
 * B*H*L*d must stay below about 8.4 million elements in LSSA/LSSAR mode).
 * No cudaMalloc, cudaFree or pool allocation is made.
 *
 * The first call on a device looks up that device's copy of the array (and
 * may make the CUDA driver load the library's device code); make that first
 * call before any stream capture.  All calls share the one array per device
 * and it keeps the previous call's contents; the parts that must start at zero
 * are cleared by each call on its stream.  Calls whose execution overlaps on
 * the GPU (different streams, or different host threads, without ordering
 * between them) race on the array: order them.  The device address of the
 * array is looked up once per device and kept: do not use the library on a
 * device after cudaDeviceReset (or any other teardown of its primary context)
 * in the same process.
 */
int lssar_attn_fwd_noalloc(const void *q, const void *k, const void *v, void *out,
                           int B, int H, int L, int d, int p, int mode, cudaStream_t stream);

/*
 * Introspection of the attention kernel's work schedule (host only, no CUDA
 * call).  Work items are pairs of 128-row Q tiles of one head, numbered
 * longest first (item i: head i % BH, pair n_pairs - 1 - i / BH).  CTA c of a
 * grid of `grid` CTAs first processes first[2c] and then first[2c+1] (-1:
 * none), then the items from *tail_base on, as a global counter hands them
 * out.  first must hold 2*grid ints; 1 <= grid <= 256.  Returns LSSAR_OK,
 * LSSAR_ERR_NULL or LSSAR_ERR_SHAPE.
 */
int lssar_schedule_plan(int BH, int n_qtiles, int grid, int *first, int *tail_base);

/*
 * The launch plan of lssar_attn_decode for these sizes on the current device
 * (host only: queries the device's SM count and occupancy, launches nothing).
 * Outputs, each may be NULL: *path = 0 (one launch, a thread-block cluster per
 * head), 1 (one cooperative launch) or 2 (three launches); *launches = the
 * kernel launches one decode call makes (1, 1 or 3); *chunks = pieces of
 * each head's cache; *chunk_rows = keys per piece (the last one shorter).
 * The environment variable LSSAR_DECODE_PATH is honoured as by the call.
 * Returns LSSAR_OK, LSSAR_ERR_SHAPE / LSSAR_ERR_HEADDIM on sizes the call
 * rejects, or LSSAR_ERR_CUDA (no device).
 */
int lssar_decode_plan(int B, int H, int L, int d, int *path, int *launches, int *chunks, int *chunk_rows);

/*
 * TEST ONLY: the failure path of the bounded waits.  Runs one decode step
 * (B=1 H=4 L=512 d=64, zero inputs, internal scratch) whose producer warps
 * withhold every copy, so that each wait of that launch gives up after its
 * 2 s bound: the kernel records decode code 41 in the device error word,
 * leaves its loops and ends without a fault (no copy is in flight).  Takes
 * about 2 s on the GPU; returns LSSAR_OK once launched, LSSAR_ERR_CUDA
 * otherwise.  Read the code with lssar_device_error_word afterwards.
 */
int lssar_selftest_stall(cudaStream_t stream);

/* Human-readable name of a status code (static string, never NULL). */
const char *lssar_status_string(int status);

/*
 * Reads and clears the device error word of the current device: 0 when no
 * kernel of this library has hit a bounded wait or a bad length, count (51) or
 * page number (52) of a paged cache since the last call, else the code (of a
 * wait: its pipeline stage, from 1 in the forward, 21 in the backward, 41 in the
 * decode step, 53 in the paged one, 61 in the paged chunk) of the first.  Synchronises
 * the current device.  Returns LSSAR_OK or LSSAR_ERR_CUDA.
 */
int lssar_device_error_word(unsigned int *word);

/* Version of this ABI: major * 10000 + minor * 100 + patch. */
int lssar_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LSSAR_ATTN_FWD_H */
