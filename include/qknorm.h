/*
 * qknorm.h -- C ABI of the MI355X (gfx950) QK-Norm library.
 *
 * QK-Norm is RMSNorm applied to the query and key parts of a fused QKV
 * projection output, in place, with the value part left untouched.
 *
 *   RMSNorm of a width-n group x with weights g:
 *       S = sum_j x_j^2,   y_j = g_j * x_j / sqrt(S / n + eps)
 *   (SwiftQK verdict page, pith.science, arXiv 2608.09160 -- core discovery
 *    and key machinery: the divisor is the square root of the full-width mean
 *    square plus eps, and the result is multiplied by the RMS weights.)
 *
 * Data layout shared by every entry point
 * ---------------------------------------
 *   qkv   fused rows [T, ld] in device memory, row-major, ld in ELEMENTS.
 *         Row t starts at element t*ld.  Columns [0, wq) are Q, [wq, wq+wk)
 *         are K, and columns >= wq+wk (V, padding) are never read or written.
 *         The row pitch ld*esize may be at most 64 MiB (QKNORM_E_UNSUPPORTED).
 *         (Lesson "Explain combined QKV projection and why it's faster than
 *         three separate projections?", section "With GQA": the fused output
 *         is Q heads, then K heads, then V heads, split by those widths.)
 *   dtype QKNORM_F32, QKNORM_BF16 or QKNORM_F16: qkv and gamma share it.
 *         QKNORM_FP8_E4M3: qkv holds OCP FP8 E4M3 values (1 sign, 4 exponent
 *         bits with bias 7, 3 fraction bits; no infinities; largest finite
 *         448), unscaled, and gamma is bf16.  (SwiftQK verdict page, Section
 *         IV-C / Fig. 2(b) and the summary: the activations are BF16 or
 *         FP8-E4M3, and error is measured at that format.)
 *         Arithmetic is fp32 throughout; each output element is rounded
 *         once, to nearest even, to the I/O dtype; FP8 results beyond +-448
 *         saturate to +-448 (a NaN stays NaN).  Partial sums are always fp32.
 *   eps   fp32, finite, >= 0; added to the mean square inside the root.
 *
 * Ownership, streams and threads
 * ------------------------------
 *   Every pointer is a device pointer owned by the caller.  The library never
 *   allocates, frees or synchronises: each call enqueues its kernels on
 *   `stream` (a hipStream_t; NULL is the null stream) and returns.  It keeps
 *   no mutable state besides a per-device cache of the compute-unit count, so
 *   calls from several host threads are safe.  gamma and partial buffers must
 *   not overlap the Q+K region being normalised.
 *
 * Errors
 * ------
 *   Every argument is checked on the host before any HIP call; on an error
 *   nothing is enqueued and a negative QKNORM_E_* code is returned.  T == 0 is
 *   a valid no-op.  A pointer may be NULL only where nothing would be read or
 *   written through it (T == 0, or the width it serves is 0).  After the
 *   launch, a HIP launch error is reported as QKNORM_E_HIP; faults during
 *   execution surface at the caller's next synchronisation, as usual for
 *   asynchronous work.  No C++ exception crosses this interface.
 */
#ifndef QKNORM_H
#define QKNORM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QKNORM_ABI_VERSION 1

/* dtype codes */
#define QKNORM_F32 0
#define QKNORM_BF16 1
#define QKNORM_F16 2
#define QKNORM_FP8_E4M3 3

/* return codes */
#define QKNORM_OK 0
#define QKNORM_E_NULLPTR -1     /* a pointer that would be used is NULL */
#define QKNORM_E_SHAPE -2       /* negative size, ld too small, shard count does not divide */
#define QKNORM_E_ALIGN -3       /* base, row pitch, head or shard not a multiple of 16 bytes */
#define QKNORM_E_DTYPE -4       /* dtype not one of the codes above */
#define QKNORM_E_UNSUPPORTED -5 /* a valid request the library does not implement (e.g. head_dim) */
#define QKNORM_E_EPS -6         /* eps negative, NaN or infinite */
#define QKNORM_E_HIP -7         /* the HIP runtime refused the launch or device query */

/*
 * Per-head QK-Norm.
 * Each Q head (hq of them, columns h*head_dim) and each K head (hkv of them,
 * columns hq*head_dim + h*head_dim) is normalised over its own head_dim
 * values.  One gamma of length head_dim serves all Q heads (gamma_q), another
 * all K heads (gamma_k).  With hkv == 0 this is a standalone [T, hq, head_dim]
 * tensor (ld = hq*head_dim) and gamma_k may be NULL.
 * (sglang PR "Add turbomind_rms_norm to accelerate QK norm in Qwen3 models",
 *  #13189, Motivation and Modifications: the QK norm is an RMSNorm whose
 *  hidden size is the head dimension, 128 in the benchmark tables.)
 *
 * Serves any RMSNorm whose width is a head (the PR routes every RMSNorm of
 * hidden size <= 128 to it): a plain [T, hidden] RMSNorm is hq = 1, hkv = 0,
 * head_dim = ld = hidden.
 *
 * Requires: head_dim*esize a multiple of 16 bytes (else QKNORM_E_ALIGN) and
 * at most 1024 bytes (FP8 head_dim 16..1024 in steps of 16, bf16/fp16 8..512
 * in steps of 8, fp32 4..256 in steps of 4); ld >= (hq+hkv)*head_dim; qkv,
 * gamma and ld*esize 16-byte aligned.  QKNORM_E_UNSUPPORTED also when one
 * launch step over the smallest heads (16 or 32 bytes) would span 2 GiB of
 * rows (a tiny head in rows of tens of MiB).
 */
int qknorm_per_head(void *qkv, int64_t T, int64_t ld, int32_t hq, int32_t hkv,
                    int32_t head_dim, const void *gamma_q, const void *gamma_k,
                    float eps, int32_t dtype, void *stream);

/*
 * Layerwise QK-Norm through shard partials, fused into one launch.
 * Q (width wq, gamma_q of length wq) and K (width wk, gamma_k of length wk)
 * are each normalised over their whole width.  The sum of squares of each is
 * taken as nshards contiguous equal shard partials in fp32, which are added
 * in shard order; the mean divides by the FULL width.  Each element is read
 * from memory once and written once while each of Q and K is at most
 * min(nshards, 8) x 4 KiB per row (bf16: 2048 values per shard-owning wave,
 * so 16384 with 8 shards, 2048 with one; FP8: not both at that limit), and
 * for FP8 also when Q is 4, 8 or 16 KiB and K a quarter or an eighth of it.
 * Wider rows take a streamed kernel that reads the row a second time to
 * apply the scale (that re-read is mostly served from L2).
 * (SwiftQK summary page, newx.sg, Abstract: the layerwise normalisation
 *  factor depends on the full hidden vector.  SwiftQK verdict page, key
 *  machinery: the per-shard factor over S_local,r is replaced by the global
 *  one over the sum of the S_local,r.)
 *
 * Requires: nshards >= 1 dividing wq and wk, nshards <= 1024; each shard
 * (wq/nshards and wk/nshards elements) a multiple of 16 bytes.  The result
 * depends on nshards only through fp32 rounding, and equals
 * qknorm_partial_sumsq followed by qknorm_apply_scalar bit for bit.
 */
int qknorm_layerwise(void *qkv, int64_t T, int64_t ld, int64_t wq, int64_t wk,
                     const void *gamma_q, const void *gamma_k, float eps,
                     int32_t nshards, int32_t dtype, void *stream);

/*
 * Phase A of the two-phase layerwise path: shard partial sums of squares.
 * part_q[r*T + t] = fp32 sum of x[t, c]^2 over Q columns
 * [r*wq/nshards, (r+1)*wq/nshards); part_k likewise over the K columns
 * (offset wq).  Layout [nshards][T], contiguous per shard -- the per-token
 * scalar each tensor-parallel rank would send.  qkv is not modified.
 * (SwiftQK verdict page, key machinery and referee major comment on
 *  Section III-B / Algorithm 1: each rank publishes its local per-token sum
 *  of squares into a buffer indexed by rank and token.)
 *
 * Requires the shard conditions of qknorm_layerwise; part_* 4-byte aligned.
 */
int qknorm_partial_sumsq(const void *qkv, int64_t T, int64_t ld, int64_t wq,
                         int64_t wk, int32_t nshards, float *part_q, float *part_k,
                         int32_t dtype, void *stream);

/*
 * Phase C of the two-phase layerwise path: combine and apply.
 * For each token t: S_q = part_q[0*T+t] + part_q[1*T+t] + ... (nparts terms,
 * in that order, fp32), scale_q = 1/sqrt(S_q/norm_wq + eps), and every Q
 * element becomes x * gamma_q[c] * scale_q (K likewise).  On one device
 * norm_wq == wq and nparts == nshards.  Under tensor parallelism a rank
 * passes its LOCAL slice (wq, wk, gamma slices), the partials gathered from
 * all ranks (nparts = ranks) and the FULL widths as norm_wq, norm_wk.
 * (SwiftQK verdict page, key machinery: the global factor divides the summed
 *  local sums of squares by the full width.)
 *
 * Requires: 1 <= nparts <= 1024; norm_wq >= wq and norm_wk >= wk (and >= 1
 * where the width is nonzero); qkv, gamma and ld*esize 16-byte aligned,
 * wq*esize and wk*esize multiples of 16 bytes.
 */
int qknorm_apply_scalar(void *qkv, int64_t T, int64_t ld, int64_t wq, int64_t wk,
                        const float *part_q, const float *part_k, int32_t nparts,
                        int64_t norm_wq, int64_t norm_wk, const void *gamma_q,
                        const void *gamma_k, float eps, int32_t dtype, void *stream);

/*
 * QKV projection with per-head QK-Norm fused into its epilogue.
 * qkv[t, n] = sum_k x[t, k] * w[n, k] for n < N = (hq + 2*hkv)*head_dim,
 * accumulated in fp32; then, unless flags has QKNORM_PROJ_PLAIN, each Q head
 * (columns h*head_dim, gamma_q) and each K head (columns hq*head_dim +
 * h*head_dim, gamma_k) of every row is normalised as by qknorm_per_head, but
 * on the fp32 accumulator before any rounding; V columns are stored as
 * computed.  One pass replaces a projection that writes qkv and a norm that
 * reads and rewrites it.
 * (Lesson "Explain combined QKV projection and why it's faster than three
 *  separate projections?", section "With GQA": one projection whose output is
 *  split into Q, K and V heads; sglang PR #13189: the QK norm is an RMSNorm
 *  over the head dimension.)
 *
 * x   [T, hidden], row pitch ldx (elements); w [N, hidden], the projection
 *     weight with one row per output column, pitch ldw; qkv [T, ld] output,
 *     columns >= N not written.  dtype QKNORM_BF16 or QKNORM_F16: x, w,
 *     gamma and qkv share it (others give QKNORM_E_UNSUPPORTED); products are
 *     accumulated in fp32 either way and rounded once, to nearest-even.
 *     flags: 0, or QKNORM_PROJ_PLAIN for the plain projection (gamma and eps
 *     unused).
 * Requires: hidden a multiple of 64 and head_dim 64, 128 or 256 (else
 * QKNORM_E_UNSUPPORTED); ldx, ldw >= hidden and ld >= N; x, w, qkv and gamma
 * 16-byte aligned, pitches*2 multiples of 16 bytes; 256 rows of x, of w and
 * of qkv each below 2 GiB.  x, w and gamma must not overlap qkv.
 */
#define QKNORM_PROJ_PLAIN 1
int qknorm_qkv_proj_per_head(const void *x, int64_t ldx, const void *w, int64_t ldw, void *qkv,
                             int64_t ld, int64_t T, int64_t hidden, int32_t hq, int32_t hkv,
                             int32_t head_dim, const void *gamma_q, const void *gamma_k,
                             float eps, int32_t flags, int32_t dtype, void *stream);

/*
 * Workspace bytes qknorm_qkv_proj_per_head_ws needs for T tokens of these
 * heads: for 1 <= T <= 64, 16*T*N bytes up to 8 tokens, 32*T*N from 9 to 32
 * and 16*T*N from 33 to 64 (N = (hq + 2*hkv)*head_dim; rounded up to a
 * multiple of 256); 0 for other T, which need none.  Negative on error:
 * QKNORM_E_SHAPE for a negative T, hq or hkv or head_dim <= 0,
 * QKNORM_E_UNSUPPORTED for T or N beyond the projection's limits.  Host only;
 * no HIP call.
 */
int64_t qknorm_qkv_proj_workspace_bytes(int64_t T, int32_t hq, int32_t hkv, int32_t head_dim);

/*
 * qknorm_qkv_proj_per_head with a workspace, for decode and other small
 * token counts.  At 1 <= T <= 64 the projection is mostly a stream over the
 * weight (N x hidden, each element read once), and the few blocks of one
 * head (or one row tile of a head) each cannot read it at the chip's rate.
 * With a workspace the weight is cut into narrow column groups by slices of
 * hidden, one block each for all T tokens, which leave fp32 partial sums in
 * the workspace; a second launch on the same stream adds each output's
 * partials in slice order, normalises each Q and K head of every row and
 * stores.
 * The result has the definition of qknorm_qkv_proj_per_head (fp32
 * accumulation, per-head QK-Norm on the fp32 sums, one rounding); the fp32
 * additions come in another order, so the two calls may differ in the last
 * bit.  For any other T the call is qknorm_qkv_proj_per_head and the
 * workspace is not used (it may be NULL).
 * (Lesson "Explain combined QKV projection and why it's faster than three
 *  separate projections?", sections "With GQA" and "Why it is faster": one
 *  projection split into Q, K and V heads; at decode sizes it is bound by
 *  memory traffic, not arithmetic.)
 *
 * workspace: device memory owned by the caller, 16-byte aligned, at least
 * qknorm_qkv_proj_workspace_bytes(T, hq, hkv, head_dim) bytes, given in
 * workspace_bytes (less: QKNORM_E_SHAPE; NULL: QKNORM_E_NULLPTR; misaligned:
 * QKNORM_E_ALIGN).  Its contents on entry do not matter and afterwards hold
 * partial sums.  It must not overlap x, w, gamma or qkv, and must not serve
 * two calls that can run at the same time (calls on different streams).
 * All other arguments and errors as for qknorm_qkv_proj_per_head.
 */
int qknorm_qkv_proj_per_head_ws(const void *x, int64_t ldx, const void *w, int64_t ldw, void *qkv,
                                int64_t ld, int64_t T, int64_t hidden, int32_t hq, int32_t hkv,
                                int32_t head_dim, const void *gamma_q, const void *gamma_k,
                                float eps, int32_t flags, int32_t dtype, void *workspace,
                                int64_t workspace_bytes, void *stream);

/*
 * qknorm_qkv_proj_per_head_ws for callers that cannot allocate a workspace
 * (code under HIP graph capture, serving loops that may not allocate,
 * harnesses that forbid it): the same kernels, with the library's own
 * scratch in place of the workspace.  The scratch is one array of 8 MiB per
 * GPU, in the library's device memory from its load until the process ends;
 * this call allocates and frees nothing.  Token counts whose workspace
 * (qknorm_qkv_proj_workspace_bytes) would exceed 8 MiB get
 * QKNORM_E_UNSUPPORTED before anything is enqueued (N up to 16384 at 16
 * tokens, up to 8192 at 32 or 64; a Qwen3-8B layer has N = 6144).  Every call on one GPU shares that GPU's scratch: calls that can
 * run at the same time on one GPU (different streams) race and must not
 * overlap.  Nothing in the scratch needs clearing between calls.  Devices
 * numbered 64 or higher get QKNORM_E_HIP.  Arguments, results and other
 * errors as for qknorm_qkv_proj_per_head_ws (for the same inputs the two
 * give the same bits).
 */
int qknorm_qkv_proj_per_head_noalloc(const void *x, int64_t ldx, const void *w, int64_t ldw,
                                     void *qkv, int64_t ld, int64_t T, int64_t hidden, int32_t hq,
                                     int32_t hkv, int32_t head_dim, const void *gamma_q,
                                     const void *gamma_k, float eps, int32_t flags, int32_t dtype,
                                     void *stream);

/*
 * ---------------------------------------------------------------------------
 * 8-bit projection and 4-bit KV cache: one attention block's serving path,
 *   qknorm_quant_rows -> qknorm_qkv_proj_quant -> qknorm_kv_append
 *   -> qknorm_kv_attention.
 * The conventions above hold (device pointers, no allocation, no
 * synchronisation, host checks, T == 0 a no-op); `dtype` is QKNORM_BF16 or
 * QKNORM_F16 unless said otherwise (others: QKNORM_E_UNSUPPORTED).  The
 * stream's device must be the current one.
 * ---------------------------------------------------------------------------
 */

/*
 * Rows to 8-bit integers with one scale a row:
 *   scale[t] = max_j |x[t,j]| / 127                      (fp32)
 *   q[t,j]   = 127 * x[t,j] / max_j |x[t,j]|, rounded to nearest, halfway to
 *              even (the exact quotient decides)
 * x [T, n] of `dtype`, pitch ldx; q [T, n] int8, pitch ldq; scale [T].  Rows
 * whose largest magnitude is below 2^-100 get zeros and scale 0; rows with an
 * infinity or a NaN get zeros and scale NaN, which makes every output that
 * uses them NaN.  A projection weight [N, hidden] quantises the same way, one
 * scale per output channel.
 * Requires: x and q 16-byte aligned, n and ldq multiples of 16, ldx of 8; T
 * below 2^24, n up to 2^24.  q and scale must not overlap x.
 */
int qknorm_quant_rows(const void *x, int64_t ldx, void *q, int64_t ldq, float *scale, int64_t T,
                         int64_t n, int32_t dtype, void *stream);

/*
 * qknorm_qkv_proj_per_head on 8-bit integers:
 *   qkv[t,n] = (sum_k x[t,k] * w[n,k]) * w_scale[n] * x_scale[t]
 * with x [T, hidden] and w [N, hidden] int8 (pitches ldx, ldw in elements),
 * x_scale [T] and w_scale [N] fp32; then per-head QK-Norm of Q and K heads
 * (unless QKNORM_PROJ_PLAIN), in fp32, one rounding to `dtype` (qkv's and
 * gamma's).  The integer sums are exact (int32); the two scales are applied in
 * the order written.
 * workspace: NULL, or device memory of workspace_bytes >=
 * qknorm_qkv_proj_quant_workspace_bytes(T, hq, hkv, head_dim), 16-byte
 * aligned, not shared by calls that can run at the same time: from 1 to 64
 * tokens the weight is then split over many more blocks (int32 partials, a
 * second launch adds them).  With and without it the integer sums are the
 * same; a normalised output may differ in its last bit.
 * Requires what qknorm_qkv_proj_per_head does, with ldx and ldw multiples of
 * 16, hidden a multiple of 64 below 131072 (no int32 sum overflows), and
 * the scales 4-byte aligned.
 */
int qknorm_qkv_proj_quant(const void *x, int64_t ldx, const float *x_scale, const void *w, int64_t ldw,
                         const float *w_scale, void *qkv, int64_t ld, int64_t T, int64_t hidden,
                         int32_t hq, int32_t hkv, int32_t head_dim, const void *gamma_q,
                         const void *gamma_k, float eps, int32_t flags, int32_t dtype,
                         void *workspace, int64_t workspace_bytes, void *stream);

/* Workspace bytes of the form above for T tokens (0: none is used). */
int64_t qknorm_qkv_proj_quant_workspace_bytes(int64_t T, int32_t hq, int32_t hkv, int32_t head_dim);

/*
 * The 4-bit KV cache.  A page holds QKNORM_KV_PAGE tokens' K and V of all
 * hkv heads: hkv blocks of 64*head_dim + 256 bytes, page p at
 * cache + p*page_stride.  A block:
 *   K codes    byte t*head_dim/2 + j: dims 2j (low 4 bits) and 2j+1 of token t
 *   V codes    byte 32*head_dim + 64*j + t: dims 2j and 2j+1 of token t
 *   K scales   bf16 at byte 64*head_dim + 2t
 *   V scales   bf16 at byte 64*head_dim + 128 + 2t
 * A code is four-bit floating point (1 sign, 2 exponent, 1 fraction bits: 0,
 * .5, 1, 1.5, 2, 3, 4, 6 and their negatives), and a value is code * scale.  One
 * scale serves one head vector of one token: scale = max|x| / 6 rounded to
 * bf16, code = x / scale rounded to nearest, halfway to the even code, at most
 * 6.  A vector below 2^-100 throughout is stored as zeros with scale 0, one
 * with an infinity or a NaN as zeros with scale NaN.
 * head_dim 64, 128 or 256 (others: QKNORM_E_UNSUPPORTED); cache and
 * page_stride (bytes, at least a page) 16-byte aligned.
 */
#define QKNORM_KV_PAGE 64

/* hkv * (64*head_dim + 256); negative on error. */
int64_t qknorm_kv_page_bytes(int32_t hkv, int32_t head_dim);

/*
 * Stores K and V of fused rows (qkv [T, ld]: hq Q heads, hkv K heads, hkv V
 * heads; K normalised already) at slots[t] = page*64 + place (int64, 8-byte
 * aligned).  A row whose slot is negative or at or past num_pages*64 is
 * skipped.  Each slot may be named once in a call: a slot named by two rows
 * ends up with bytes of either.
 */
int qknorm_kv_append(const void *qkv, int64_t T, int64_t ld, int32_t hq, int32_t hkv,
                      int32_t head_dim, void *cache, int64_t num_pages, int64_t page_stride,
                      const int64_t *slots, int32_t dtype, void *stream);

/*
 * The values held at slots[t] into k[t, h*head_dim + d] and v (pitches ldk,
 * ldv; dtype QKNORM_F32, QKNORM_BF16 or QKNORM_F16): code * scale, rounded
 * once.  Rows whose slot names no place are left as they are.  Slots may
 * repeat.  k, v 16-byte aligned, pitches multiples of 16 bytes.
 */
int qknorm_kv_gather(const void *cache, int64_t num_pages, int64_t page_stride, const int64_t *slots,
                      int64_t T, int32_t hkv, int32_t head_dim, void *k, int64_t ldk, void *v,
                      int64_t ldv, int32_t dtype, void *stream);

/*
 * Causal attention of fused rows' Q heads over the 4-bit cache.
 * Sequence b has seq_lens[b] tokens in the cache, token j at place j%64 of
 * page page_table[b*table_stride + j/64] (entries past its length are not
 * read).  Its rows are q_starts[b] .. q_starts[b+1]-1 of the T rows, its last
 * tokens, already in the cache (q_starts NULL: T == B and row b alone): row i
 * of n is token p = seq_lens[b] - n + i and sees tokens 0..p, with window > 0
 * only p-window+1..p.  Query head h reads KV head h / (hq/hkv).
 *   out[t,h,:] = sum_j softmax_j(scale * q.K_j) V_j,
 *   lse[t,h]   = log sum_j exp(scale * q.K_j)        (NULL: not wanted)
 * Scores are fp32 (products beyond its range are infinite); a visible token
 * whose K, V or Q holds a NaN makes the row NaN, as the formula does.
 * A row that sees no token gets zeros and lse = -infinity.  Rows of no
 * sequence (before q_starts[0], past q_starts[B]) are left as they are.
 * A page number outside [0, num_pages) hides its tokens.  Hidden tokens and
 * what lies past a sequence's length may hold anything.  Softmax statistics and
 * sums are fp32; weights are rounded to fp16 (11 bits) for the product with V.
 * seq_lens and q_starts are read on the GPU (a captured graph may be replayed
 * with others); lengths are taken within [0, 64*max_pages], row offsets within
 * [0, T]; offsets must not decrease (else the rows concerned are undefined).
 *
 * qkv [T, ld] and out [T, ldo] (hq*head_dim columns used) 16-byte aligned,
 * pitches multiples of 8 elements, ldo at most 32 MiB; other arrays 4-byte
 * aligned; hq a multiple of hkv; scale finite (QKNORM_E_SHAPE); B <= 4096.
 * out, lse and workspace must not overlap the inputs.  workspace: 16-byte
 * aligned, at least
 * qknorm_kv_attention_workspace_bytes(T, B, max_pages, hq, hkv, head_dim)
 * bytes, contents irrelevant on entry, not shared by calls that can run at the
 * same time (replays of two captured graphs included).
 */
int qknorm_kv_attention(const void *qkv, int64_t T, int64_t ld, const void *cache, int64_t num_pages,
                         int64_t page_stride, const int32_t *page_table, int64_t table_stride,
                         int64_t max_pages, const int32_t *seq_lens, const int32_t *q_starts, int64_t B,
                         void *out, int64_t ldo, float *lse, int32_t hq, int32_t hkv, int32_t head_dim,
                         float scale, int32_t window, int32_t dtype, void *workspace,
                         int64_t workspace_bytes, void *stream);
int64_t qknorm_kv_attention_workspace_bytes(int64_t T, int64_t B, int64_t max_pages, int32_t hq,
                                             int32_t hkv, int32_t head_dim);

/* Static description of a return code; never NULL. */
const char *qknorm_strerror(int code);

/* QKNORM_ABI_VERSION of the built library. */
int qknorm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QKNORM_H */
