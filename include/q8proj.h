/*
 * q8proj.h -- C ABI of the GB300 (sm_103a) int8 quantized projection library
 * (libq8proj.so).
 *
 * The path: an f32 activation is encoded once into a q8_0 "plane", either by a
 * standalone quantizer or by the producer kernel that computes it (RMSNorm or
 * SwiGLU), and that plane is contracted with Q8_0 weights by a batch-1 GEMV
 * (decode) or a GEMM (prefill).  For a decode token the encoding can also
 * happen inside the GEMV launch that consumes it (q8_0_gemv_fused), and the
 * gate/up GEMV can write the SwiGLU output's plane itself (q8_0_gemv_gate_up).
 *
 * Formats
 *   Q8_0 weight block: 34 bytes -- little-endian f16 scale d at +0, then 32
 *     int8 values at +2.  A weight matrix of n rows and k columns is n rows of
 *     k/32 consecutive blocks (row pitch 34*k/32 bytes), with no padding.
 *     ("Part 4 - Lecture 05 - Fusion and the Activation-Quantization
 *     Discipline", sec. 2.1.)
 *   q8_0 activation plane: per token row t and 32-element block b,
 *       qs[t*k + 32*b + j]  int8, j = 0..31
 *       ds[t*(k/32) + b]    uint32: f16 bits of d in bits 0..15, the int16
 *                           block sum ssum = sum_j q_j in bits 16..31
 *     with d = amax/127 (computed in f32), q = rint(x * (1/d)) clamped to
 *     [-127, 127], d stored rounded to f16.  The plane has rows_pad >= rows
 *     rows; rows rows..rows_pad-1 are written as zeros.
 *     ("54 - r51 - producer-fused A-quantize mode 1", sec. 2.1 and 3.1.)
 *
 * Conventions for every entry point
 *   - All data pointers are DEVICE pointers owned by the caller; the library
 *     never allocates, frees or caches device memory between calls.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Work is enqueued asynchronously; the call returns before the
 *     GPU finishes.  Errors that only the GPU can detect (a bounded wait that
 *     ran out) are reported by q8_check().
 *   - Outputs are overwritten, never accumulated into, and must not alias
 *     any input.
 *   - Sizes are int64_t element counts; k must be a positive multiple of 32.
 *   - Pointers must be 16-byte aligned (Q8_ERR_ALIGN otherwise).
 *   - The return value is a status code (Q8_OK = 0).  On a non-zero return
 *     nothing was enqueued.  There is no fallback path: a rejected shape is
 *     an error, not a slow path.
 */
#ifndef Q8PROJ_H
#define Q8PROJ_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define Q8_API __attribute__((visibility("default")))
#else
#define Q8_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define Q8_OK                 0
#define Q8_ERR_ARG            1  /* NULL pointer, non-positive or inconsistent size, k % 32 != 0 */
#define Q8_ERR_ALIGN          2  /* a pointer is not 16-byte aligned */
#define Q8_ERR_DEVICE         3  /* current device is not sm_103 (GB300) or cannot be queried */
#define Q8_ERR_LAUNCH         4  /* the kernel launch failed (cudaGetLastError) */
#define Q8_ERR_DEVICE_TIMEOUT 5  /* a bounded on-device wait ran out (reported by q8_check) */
#define Q8_ERR_CUDA           6  /* another CUDA runtime error (stream sync, symbol copy) */
#define Q8_ERR_TOO_BIG        7  /* the request needs more than the fixed scratch of q8_0_gemm_noalloc */
#define Q8_ERR_DATA           8  /* a length, page, slot, parent, path, offset, row or place read on the device is out of range (reported by q8_check) */

/* Recommended number of plane rows for `rows` tokens: rows rounded up to a
 * multiple of 128 (the GEMM's token tile).  Any rows_pad >= rows is accepted
 * by every entry point; this is a convenience only. */
Q8_API int64_t q8_plane_rows(int64_t rows);

/* Human-readable name of a status code (static storage; never NULL). */
Q8_API const char *q8_strerror(int status);

/*
 * quantize_q8_0 -- standalone q8_0 quantizer (the "prepass").
 *   x   : f32 [rows][k] row-major (input)
 *   qs  : int8 [rows_pad][k] (output plane values)
 *   ds  : uint32 [rows_pad][k/32] (output packed d | ssum)
 * rows >= 0 (rows = 0 only zero-fills), rows_pad >= max(rows, 1), k % 32 == 0.
 * Defined by the quantize body of "54 - r51 - producer-fused A-quantize
 * mode 1", sec. 3.2, and the zero tail of sec. 3.1.
 */
Q8_API int quantize_q8_0(const float *x, int64_t rows, int64_t k,
                  int8_t *qs, uint32_t *ds, int64_t rows_pad, void *stream);

/*
 * rmsnorm_quant -- RMSNorm fused with q8_0 quantization of its output.
 *   x   : f32 [rows][d] (input)       w : f32 [d] (input weight)
 *   y   : f32 [rows][d] (output, y = (x * rsqrt(mean(x^2) + eps)) * w), or
 *         NULL when y is dead -- every consumer reads the plane -- and only
 *         the plane is written ("mode 2", the sequel that "54 - r51 -
 *         producer-fused A-quantize mode 1" sec. 5 points to: the f32 write
 *         and its re-read are what is left to remove).
 *   qs, ds : plane of y with rows_pad rows (output); the plane is exactly the
 *            q8_0 encoding of the f32 values y holds (or would hold), the
 *            same bytes whether y is written or not.
 * d % 32 == 0, d <= 32768 (the row is held in registers), rows >= 0,
 * rows_pad >= max(rows, 1).
 * "54 - r51 - producer-fused A-quantize mode 1", sec. 2.3 and 3.2
 * (rms_norm_quant_f32_t: one pass writes y and the plane).
 */
Q8_API int rmsnorm_quant(const float *x, const float *w, float eps, float *y,
                  int64_t rows, int64_t d,
                  int8_t *qs, uint32_t *ds, int64_t rows_pad, void *stream);

/*
 * swiglu_quant -- SwiGLU fused with q8_0 quantization of its output.
 *   gate, up : f32 [rows][nf] (inputs)
 *   y        : f32 [rows][nf] (output, y = gate / (1 + exp(-gate)) * up), or
 *              NULL when y is dead (mode 2, as for rmsnorm_quant): 4 of the
 *              13.125 bytes per element this call moves are that write.
 *   qs, ds   : plane of y (output), exactly the q8_0 encoding of y, the same
 *              bytes whether y is written or not.
 * nf % 32 == 0, rows >= 0, rows_pad >= max(rows, 1).
 * "54 - r51 - producer-fused A-quantize mode 1", sec. 3.2
 * (swiglu_quant_f32_t).
 */
Q8_API int swiglu_quant(const float *gate, const float *up, float *y,
                 int64_t rows, int64_t nf,
                 int8_t *qs, uint32_t *ds, int64_t rows_pad, void *stream);

/*
 * q8_0_gemv -- batch-1 projection y[i] = sum_b d_w(i,b) * d_a(b) * sum_j qw*qa.
 *   w      : n rows of k/32 Q8_0 blocks (input, 16-byte aligned base)
 *   qs, ds : plane row 0 (input; only row 0 is read)
 *   y      : f32 [n] (output)
 * n >= 1, k % 32 == 0.  Row grouping and the split of k across warps are
 * chosen from (n, k) alone, deterministically; results are run-to-run
 * identical.  "Part 4 - Lecture 05", sec. 2.1-2.4.
 * The kernel is launched with programmatic dependent launch: it may start
 * streaming `w` while the kernel enqueued just before it on `stream` is
 * still running, and reads the plane only after that kernel has finished.
 * `w` (the model weights) must therefore not be written by the kernel
 * immediately preceding the call on the same stream.
 */
Q8_API int q8_0_gemv(const void *w, int64_t n, int64_t k,
              const int8_t *qs, const uint32_t *ds, float *y, void *stream);

/*
 * q8_0_gemv_grouped -- several batch-1 projections of ONE activation in one
 * launch: for each i < count, projs[i].y[r] = sum_b d_w * d_a * isum over the
 * rows of projs[i].w, all against plane row 0 of (qs, ds) with the same k.
 *   projs : host array of `count` descriptors (read during the call only);
 *           each w and y is a device pointer as for q8_0_gemv, n >= 1.
 *   count : 1..Q8_MAX_GROUP.
 * Rows of all projections are spread over the whole GPU together, so small
 * projections ride along with large ones instead of each paying a launch and
 * a partly idle grid.  Same numerics as q8_0_gemv (one row is always computed
 * the same way), and the same programmatic-dependent-launch precondition on w.
 * "Part 4 - Lecture 05", sec. 2.5 (one launch for the consumers of one
 * activation) and sec. 6 (generalised to projections of different widths).
 * When (k/32) % 8 != 0 the projections are launched one by one.
 */
#define Q8_MAX_GROUP 8
typedef struct q8_gemv_proj {
    const void *w;   /* n rows of k/32 Q8_0 blocks */
    int64_t n;       /* rows (outputs) */
    float *y;        /* f32 [n] output */
} q8_gemv_proj;

Q8_API int q8_0_gemv_grouped(const q8_gemv_proj *projs, int count, int64_t k,
                             const int8_t *qs, const uint32_t *ds, void *stream);

/*
 * q8_0_gemv_fused -- q8_0_gemv_grouped with its one-row producer in the same
 * launch: every CTA computes the producer's f32 row and its q8_0 encoding
 * straight into the shared memory it would otherwise fill from a plane, so
 * the producer's launch, the plane's write and re-read, and the hand-off
 * between two launches disappear.
 *   producer : Q8_PRODUCER_QUANT    a = x f32 [k]            (as quantize_q8_0)
 *              Q8_PRODUCER_RMSNORM  a = x f32 [k], norm_w = w f32 [k], eps
 *                                   (as rmsnorm_quant)
 *              Q8_PRODUCER_SWIGLU   a = gate f32 [k], b = up f32 [k]
 *                                   (as swiglu_quant)
 *              unused pointers may be NULL; all inputs are read only.
 *   projs, count, k : as for q8_0_gemv_grouped; each projs[i].y is written.
 * Result: bit for bit what the standalone producer (one row, rows_pad at most
 * the SM count -- e.g. q8_plane_rows(1)) followed by q8_0_gemv_grouped on its
 * plane returns: the producer arithmetic is one implementation shared by both
 * paths, and for RMSNorm the row's sum of squares is formed in the standalone
 * kernel's order.  No f32 row or plane is written.
 * Requires (k/32) % 8 == 0 and k <= 65536 (the staged path), k <= 32768 for
 * RMSNorm; otherwise Q8_ERR_ARG (run the producer and the GEMV as two calls).
 * Pointers 16-byte aligned (Q8_ERR_ALIGN).  The producer's inputs are read
 * only after the kernel enqueued before the call on `stream` has finished
 * (the same programmatic-dependent-launch rule as q8_0_gemv: the weights may
 * be streamed earlier); the outputs must not overlap the inputs.
 * "Part 4 - Lecture 05", sec. 3 (a one-row quantize costs a launch, not
 * bandwidth) and sec. 4 (its rule: make producer and consumer one launch, and
 * keep one implementation for the fused and the unfused path).
 */
#define Q8_PRODUCER_QUANT   1
#define Q8_PRODUCER_RMSNORM 2
#define Q8_PRODUCER_SWIGLU  3
Q8_API int q8_0_gemv_fused(const q8_gemv_proj *projs, int count, int64_t k, int producer,
                           const float *a, const float *b, const float *norm_w, float eps,
                           void *stream);

/*
 * q8_0_gemv_gate_up -- the gate and up projections of one token with SwiGLU
 * and its q8_0 encoding in the same launch: gate = Wg.x, up = Wu.x (x from
 * plane row 0 of (qs, ds), or produced in the launch as for q8_0_gemv_fused),
 * and the plane row of silu(gate) * up written straight to (qs_out, ds_out)
 * -- the input of the down projection -- with no f32 SwiGLU output and no
 * separate SwiGLU launch.  Row r of gate and row r of up are computed by the
 * same CTA; the warp that completes the 32 rows of a block encodes it.
 *   w_gate, w_up : nf rows of k/32 Q8_0 blocks each (inputs)
 *   qs, ds       : activation plane row 0 when producer == 0, else unused
 *   producer     : 0, Q8_PRODUCER_QUANT (a = x) or Q8_PRODUCER_RMSNORM
 *                  (a = x, norm_w, eps), as for q8_0_gemv_fused
 *   y_gate, y_up : f32 [nf] outputs, or NULL when not wanted
 *   qs_out       : int8 [nf], ds_out : uint32 [nf/32] -- one plane row (row 0
 *                  of a plane; other rows are not touched)
 * Result: y_gate / y_up bit for bit as q8_0_gemv_grouped (or _fused) writes
 * them, and the plane bit for bit as swiglu_quant writes it for those values
 * (the same SwiGLU and encoding arithmetic).
 * Requires nf % 32 == 0, (k/32) % 8 == 0, 2048 < k <= 65536 (whole rows per
 * warp on the staged path), k <= 32768 for RMSNorm; otherwise Q8_ERR_ARG.
 * Pointers 16-byte aligned (Q8_ERR_ALIGN).  The same programmatic-dependent-
 * launch rule as q8_0_gemv; outputs must not overlap inputs.
 * "54 - r51 - producer-fused A-quantize mode 1", sec. 3.2 (swiglu_quant_f32_t:
 * SwiGLU and the quantize of its output in one pass) and sec. 6 (consume the
 * data where it is hottest: here the registers of the gate/up GEMV); "Part 4 -
 * Lecture 05", sec. 4 (one launch instead of a buffer passed between two).
 */
Q8_API int q8_0_gemv_gate_up(const void *w_gate, const void *w_up, int64_t nf, int64_t k,
                             const int8_t *qs, const uint32_t *ds,
                             int producer, const float *a, const float *norm_w, float eps,
                             float *y_gate, float *y_up, int8_t *qs_out, uint32_t *ds_out,
                             void *stream);

/*
 * q8_0_gemv_batched -- the projection for a few tokens at once (decode over
 * a small batch of sequences): Y[t][i] = sum_b d_w(i,b) * d_a(t,b) * isum for
 * plane rows t < tokens, reading the weights from memory once for all of
 * them.  The formula is the GEMM's ("12 - r5-r6 re-ranking + structural
 * rewrite spec", sec. 2); the pages build only its two ends, the batch-1 GEMV
 * and the prefill GEMM, and this entry point fills the range between them.
 *   w      : n rows of k/32 Q8_0 blocks (input, 16-byte aligned)
 *   qs, ds : plane with at least `tokens` rows (input; rows >= tokens are
 *            not read)
 *   y      : f32 [tokens][n] row-major (output, overwritten)
 * 1 <= tokens <= Q8_GEMV_MAX_TOKENS, n >= 1, k % 32 == 0.  When
 * (k/32) % 8 == 0 the block dot products run on the tensor cores (int8 codes
 * widened exactly to f16, f32 accumulation of an exact integer) and each
 * block adds (d_w * d_a) * isum to one of four partial sums over k, which are
 * added in a fixed order: results are run-to-run identical.  Other k use the
 * generic kernel (weights read once per token).  Programmatic dependent
 * launch, with the same precondition on w as q8_0_gemv.
 * q8_0_gemm hands calls with t <= Q8_GEMV_MAX_TOKENS to this path (t == 1 to
 * q8_0_gemv), and calls with Q8_GEMV_MAX_TOKENS < t <= 64 to this path over
 * consecutive 16-token slices of the plane (each slice streams the weights
 * again; up to four passes cost less than the GEMM's pre-pass).
 */
#define Q8_GEMV_MAX_TOKENS 16
Q8_API int q8_0_gemv_batched(const void *w, int64_t n, int64_t k,
                             const int8_t *qs, const uint32_t *ds, int64_t tokens,
                             float *y, void *stream);

/*
 * q8_0_gemv_batched_grouped -- q8_0_gemv_batched for several projections of
 * the same activation rows in one launch: for each i < count,
 *     projs[i].y[t][r] = sum_b d_w(r,b) * d_a(t,b) * isum   (t < tokens)
 * over the rows of projs[i].w, all with the same k and plane.
 *   projs : host array of `count` descriptors (read during the call only);
 *           w and y are device pointers (16-byte aligned); y is f32
 *           [tokens][projs[i].n] row-major.
 *   count : 1..Q8_MAX_GROUP.
 *   qs, ds, tokens : as for q8_0_gemv_batched.
 * The projections' 128-row tiles form one grid, so a narrow projection (a
 * K or V of grouped-query attention) rides along with a wide one instead of
 * paying its own launch and a partly idle GPU.  The per-block arithmetic is
 * q8_0_gemv_batched's; the number of CTAs that split k for one tile (1..8) is
 * chosen from the launch's total tile count, so the partial sums over k may
 * be grouped differently than in a single call of one projection (equal bit
 * for bit where that number is the same).  Results are run-to-run identical.
 * When (k/32) % 8 != 0 the projections run one by one on the generic kernel.
 * Errors: Q8_ERR_ARG (count, shape, tokens, a NULL pointer), Q8_ERR_ALIGN,
 * Q8_ERR_DEVICE, Q8_ERR_LAUNCH.  Programmatic dependent launch as for
 * q8_0_gemv.  "Part 4 - Lecture 05", sec. 2.5 (one launch for the consumers
 * of one activation), applied to the small-batch formula above.
 */
Q8_API int q8_0_gemv_batched_grouped(const q8_gemv_proj *projs, int count, int64_t k,
                                     const int8_t *qs, const uint32_t *ds, int64_t tokens,
                                     void *stream);

/*
 * q4a_gemv -- batch-1 projection with asymmetric 4-bit weight blocks, the
 * consumer of the plane's int16 block sums:
 *     y[i] = sum_b ( d*d_a * sum_e nib_e*q_e  -  m*d_a * ssum_b ).
 * The weight value d*nib - m is the q4_K form d*s*nib - dmin*m of "12 - r5-r6
 * re-ranking + structural rewrite spec" (sec. 3) with one f16 scale and one
 * f16 min per 32 elements, and its min term takes the plane's ssum instead
 * of a second dot product, the use "54 - r51 - producer-fused A-quantize
 * mode 1" (sec. 2.1) gives the int16 field.
 *   w      : n rows of k/32 20-byte blocks (input, 16-byte aligned): f16 d at
 *            +0, f16 m at +2, then byte j (j < 16) holds element j in its low
 *            nibble and element j + 16 in its high nibble (unsigned 0..15).
 *   qs, ds : plane row 0 (input; only row 0 is read)
 *   y      : f32 [n] (output)
 * n >= 1, k % 128 == 0 (16-byte aligned rows of whole 4-block chunks),
 * k <= 206592 (the activation is staged in shared memory).  Per block two
 * fmas, d*d_a*isum then -m*d_a*ssum (both scale products exact in f32); the
 * split of a row over lanes depends on k only: results are run-to-run
 * identical.  Programmatic dependent launch: the plane is read only after the
 * kernel enqueued before it on `stream` has finished.
 */
Q8_API int q4a_gemv(const void *w, int64_t n, int64_t k,
                    const int8_t *qs, const uint32_t *ds, float *y, void *stream);

/*
 * q4a_gemv_batched -- the asymmetric 4-bit projection for a few tokens at
 * once, the weights streamed from HBM once for all of them:
 *     Y[t][i] = sum_b ( d*d_a(t,b) * sum_e nib_e*q_e(t)  -  m*d_a(t,b) * ssum(t,b) )
 * for tokens t < `tokens`.  Same weight blocks as q4a_gemv.
 *   qs, ds : plane rows 0..tokens-1 (input; rows at and past `tokens` are not
 *            read)
 *   y      : f32 [tokens][n] (output)
 * 1 <= tokens <= Q8_GEMV_MAX_TOKENS; k % 256 == 0 (8-block row pieces);
 * tokens == 1 runs q4a_gemv.  Per block: the exact integer dot of the nibbles
 * with the codes, then fma(d*d_a, isum) and fma(-(m*d_a), ssum) (scale
 * products exact in f32).  Partial sums over k are added in a fixed order:
 * results are run-to-run identical.  Errors: Q8_ERR_ARG (shape, tokens),
 * Q8_ERR_ALIGN (a pointer not 16-byte aligned), Q8_ERR_DEVICE (not sm_103),
 * Q8_ERR_LAUNCH.  Programmatic dependent launch as for q4a_gemv.
 */
Q8_API int q4a_gemv_batched(const void *w, int64_t n, int64_t k,
                            const int8_t *qs, const uint32_t *ds, int64_t tokens,
                            float *y, void *stream);

/*
 * q4a_gemv_batched_grouped -- q4a_gemv_batched for up to Q8_MAX_GROUP
 * projections of the same plane rows, as q8_0_gemv_batched_grouped is for
 * Q8_0 weights: projs[i].w holds projs[i].n rows of the 20-byte asymmetric
 * blocks, projs[i].y is f32 [tokens][projs[i].n]; k % 256 == 0, 1 <= tokens
 * <= Q8_GEMV_MAX_TOKENS.  For tokens >= 2 the projections' row tiles form one
 * launch of the small-batch kernel (per block the arithmetic of
 * q4a_gemv_batched; the number of CTAs splitting k follows the launch's total
 * tile count, so partial sums may be grouped differently than in a single
 * call, bit for bit equal where that number is the same); tokens == 1 runs
 * q4a_gemv projection by projection.  Errors as q4a_gemv_batched, plus
 * Q8_ERR_ARG for count outside 1..Q8_MAX_GROUP or a NULL descriptor.
 */
Q8_API int q4a_gemv_batched_grouped(const q8_gemv_proj *projs, int count, int64_t k,
                                    const int8_t *qs, const uint32_t *ds, int64_t tokens,
                                    void *stream);

/*
 * q8_0_gemm_workspace_bytes -- device workspace q8_0_gemm needs for n weight
 * rows, t tokens and width k: the weight codes as f16 (n*k*2 bytes), the
 * activation codes as f16 (t*k*2), and both sides' block scales as f32
 * (k/32 * 4 bytes per weight row and per token, rows and tokens rounded up to
 * the GEMM's 128 x 192 tiles), each part starting on a 1 KiB boundary; when
 * the tiles would leave most SMs idle (few weight rows or tokens) k is split
 * over up to 12 CTAs per tile and the workspace also holds their f32 partial
 * outputs (splits * t * n * 4 bytes, added in a fixed order by a reduction
 * kernel; splits * tiles <= 152, so at most about 15 MB).  The size depends
 * on (n, t, k) only.  0 when (k/32) % 8 != 0 or t <= 64 (those calls run
 * the generic or small-batch kernels and need none).
 */
Q8_API size_t q8_0_gemm_workspace_bytes(int64_t n, int64_t t, int64_t k);

/*
 * q8_0_gemm -- prefill projection Y[t][i] = sum_b d_w(i,b) * d_a(t,b) * isum.
 *   w      : n rows of k/32 Q8_0 blocks (input)
 *   qs, ds : plane with rows_pad >= t rows (input; rows >= t are not read)
 *   y      : f32 [t][n] row-major (output)
 *   workspace, workspace_bytes : caller-owned device scratch of at least
 *            q8_0_gemm_workspace_bytes(n, t, k) bytes, 16-byte aligned; its
 *            contents on entry are ignored and on return are unspecified.
 *            Two calls may share a workspace only if they are ordered on one
 *            stream.  May be NULL when that size is 0.
 * n >= 1, t >= 1, k % 32 == 0.  Every 32-wide k block is one q8_0 block on
 * both sides, so its integer dot product is scaled by d_w * d_a once.
 * Dispatch by shape: t == 1 -> q8_0_gemv; (k/32) % 8 != 0 -> the generic
 * kernel; t <= 64 -> q8_0_gemv_batched's kernel (over 16-token slices above
 * 16 tokens); otherwise the call enqueues two pre-passes that write the
 * weight codes and the plane's codes as f16 (exact) and both sides' block
 * scales as f32 into the workspace, then the tcgen05 GEMM (split over k when
 * its tiles alone would leave most SMs idle, with a reduction kernel after
 * it), all with programmatic dependent launch and the same precondition on w
 * as q8_0_gemv.
 * "12 - r5-r6 re-ranking + structural rewrite spec", sec. 2 and 3.1;
 * "54 - r51 - producer-fused A-quantize mode 1", sec. 2.1.
 */
Q8_API int q8_0_gemm(const void *w, int64_t n, int64_t k,
                     const int8_t *qs, const uint32_t *ds, int64_t t, int64_t rows_pad,
                     float *y, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Prepared weights for the prefill GEMM.  A model's weights do not change
 * between calls, so the weight pre-pass that q8_0_gemm enqueues on every
 * call (the codes widened to f16 exactly, d_w as f32 in the epilogue's
 * order) can run once per matrix instead:
 *
 * q8_0_gemm_prepared_weights_bytes -- size of the prepared form of an n x k
 * Q8_0 matrix: n*k*2 bytes of f16 codes and k/32*4 bytes of d_w per weight
 * row (rows rounded up to the GEMM's 128-row tiles), each part starting on a
 * 1 KiB boundary.  0 when (k/32) % 8 != 0 or the shape is past the GEMM's
 * grid limits (n > 65535*128, k > 2^30).
 *
 * q8_0_gemm_prepare_weights -- write that form of w into wprep (caller-owned
 * device memory of at least q8_0_gemm_prepared_weights_bytes(n, k) bytes,
 * 16-byte aligned; its layout is private to this library and valid for this
 * (n, k) only).  One kernel, enqueued on `stream` with programmatic dependent
 * launch.  Q8_ERR_ARG for a NULL pointer, a short buffer or a shape the GEMM
 * does not take, Q8_ERR_ALIGN for misaligned pointers.
 *
 * q8_0_gemm_prepared_workspace_bytes -- device workspace q8_0_gemm_prepared
 * needs: q8_0_gemm_workspace_bytes without the two weight parts.  0 when the
 * call takes a path that needs none (t <= 64 or (k/32) % 8 != 0).
 *
 * q8_0_gemm_prepared -- q8_0_gemm whose tcgen05 path reads prepared weights:
 * the same result, bit for bit, as q8_0_gemm(w, ...) (the same kernels on
 * the same operands), without the per-call weight pre-pass.
 *   w      : the Q8_0 matrix, read by the paths for t <= 64 and for
 *            (k/32) % 8 != 0; may be NULL when the call takes the tcgen05
 *            path (t > 64 and (k/32) % 8 == 0)
 *   wprep  : q8_0_gemm_prepare_weights(w, n, k, ...)'s output, read by the
 *            tcgen05 path (may be NULL otherwise).  Written earlier on this
 *            stream, or ordered before this call by the caller.
 *   qs, ds, t, rows_pad, y : as for q8_0_gemm
 *   workspace, workspace_bytes : at least
 *            q8_0_gemm_prepared_workspace_bytes(n, t, k) bytes, as for
 *            q8_0_gemm
 * "12 - r5-r6 re-ranking + structural rewrite spec", sec. 2 and 3.1 (the
 * per-block scale correction); "54 - r51 - producer-fused A-quantize mode 1",
 * sec. 2.1 (the plane).
 */
Q8_API size_t q8_0_gemm_prepared_weights_bytes(int64_t n, int64_t k);
Q8_API int q8_0_gemm_prepare_weights(const void *w, int64_t n, int64_t k,
                                     void *wprep, size_t wprep_bytes, void *stream);
Q8_API size_t q8_0_gemm_prepared_workspace_bytes(int64_t n, int64_t t, int64_t k);
Q8_API int q8_0_gemm_prepared(const void *w, const void *wprep, int64_t n, int64_t k,
                              const int8_t *qs, const uint32_t *ds, int64_t t, int64_t rows_pad,
                              float *y, void *workspace, size_t workspace_bytes, void *stream);

/*
 * q8_0_gemm_noalloc -- q8_0_gemm without a workspace argument, for callers
 * that cannot allocate device memory at this point: a serving engine that
 * handed all of the GPU's memory to its own pool at start-up, a plugin whose
 * host application forbids allocation after initialisation, or a
 * latency-critical path that cannot pay for cudaMalloc's implicit device
 * synchronisation.  The pages have no counterpart of this entry point; it
 * exists for those callers only.
 *   Arguments, results and numerics are those of q8_0_gemm (same kernels).
 *   The scratch q8_0_gemm takes from `workspace` comes instead from a 32 MiB
 *   array that is part of this library's device code
 *   (q8_0_gemm_noalloc_max_bytes()).  Every GPU that loads the library's GEMM
 *   code holds those 32 MiB until the process exits.  A request whose
 *   q8_0_gemm_workspace_bytes(n, t, k) exceeds it returns Q8_ERR_TOO_BIG
 *   (the f16 copies of both operands must fit: small projections, or t <= 64
 *   which needs no scratch at all).
 *   The entry point itself calls no cudaMalloc/cudaFree or allocating
 *   routine.  Its first call on a device looks up that device's address of
 *   the array (cudaGetSymbolAddress, with the device current), and so does
 *   the first call after the device's context has been replaced (for
 *   instance by cudaDeviceReset); make those calls before any stream capture.
 *   All calls share the one array and it keeps the last call's contents;
 *   nothing in it needs to start at zero (each call rewrites every byte it
 *   reads), but calls that overlap on the GPU -- different streams, or
 *   different host threads -- race on it and give undefined results.
 */
Q8_API int q8_0_gemm_noalloc(const void *w, int64_t n, int64_t k,
                             const int8_t *qs, const uint32_t *ds, int64_t t, int64_t rows_pad,
                             float *y, void *stream);

/* Size in bytes of the fixed scratch behind q8_0_gemm_noalloc. */
Q8_API size_t q8_0_gemm_noalloc_max_bytes(void);

/*
 * q8_0_gemm_mma -- the same contraction as q8_0_gemm on the warp-level int8
 * tensor instruction (mma.sync.m16n8k32.s8) instead of tcgen05: the legacy
 * tensor path, kept as an exact A/B baseline for q8_0_gemm.  Requires
 * (k/32) % 8 == 0 (Q8_ERR_ARG otherwise); arguments as q8_0_gemm.
 */
Q8_API int q8_0_gemm_mma(const void *w, int64_t n, int64_t k,
                         const int8_t *qs, const uint32_t *ds, int64_t t, int64_t rows_pad,
                         float *y, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Paged key/value cache and the attention that reads it: the step between the
 * q/k/v projections and the o projection, for single tokens, for trees of
 * drafted tokens that a batch-of-tokens step verifies, and for prompts.
 *
 * A sequence holds `cached` tokens from earlier steps and gets `fresh` new
 * ones in this step.  Token `pos` of sequence b lives in page
 * table[b][pos / page_size], at offset pos % page_size.  The fresh rows of all
 * sequences lie one after another: those of sequence b are rows
 * starts[b] .. starts[b + 1] - 1 of q, k, v, y, slots, masks and positions.
 *
 * The lengths, tables and masks are device data, so one captured graph serves
 * every step of the same capacity.  The free list is the host's: q8_kv_plan hands
 * out pages from its start and takes none off it, so after a step that opened
 * pages (needed > 0) the next one needs a list without them, in the same 16-byte
 * aligned buffer for a graph.  The kernels check each value they read
 * before it becomes an address: a sequence or slot that is out of range is
 * skipped (its outputs keep what they held) and q8_check reports Q8_ERR_DATA.
 * ---------------------------------------------------------------------------
 */
#define Q8_KV_F16  1   /* k, v hold f16 values */
#define Q8_KV_INT8 2   /* k, v hold int8 codes; k_scale, v_scale one f32 per (token, head): value = code * scale */
#define Q8_TREE_MAX_NODES 64   /* drafted tokens of a sequence with tree masks (one 64-bit word per token) */
#define Q8_KV_MAX_BATCH 4096   /* sequences of one call */

typedef struct q8_kv_cache {
    void *k, *v;              /* [layers][n_pages][kv_heads][page_size][head_dim] */
    float *k_scale, *v_scale; /* [layers][n_pages][kv_heads][page_size] for Q8_KV_INT8, else NULL */
    int64_t layers, n_pages;
    int32_t kv_heads;         /* 1 .. 1024 */
    int32_t page_size;        /* tokens per page, a multiple of 16 */
    int32_t head_dim;         /* 64 or 128 */
    int32_t dtype;            /* Q8_KV_F16 or Q8_KV_INT8 */
} q8_kv_cache;
/* n_pages * kv_heads * page_size < 2^31.  A page's tokens of one head are
 * contiguous, so attention streams whole 16-token rows of a head. */

/*
 * q8_kv_plan -- the integers of one step, from the request lengths.
 *   cached, fresh : int32 [batch] (inputs)
 *   held          : int32 [batch] (input) pages each table row holds already,
 *                   or NULL for ceil(cached / page_size).  They differ after
 *                   q8_kv_accept kept fewer tokens than the step had pages for.
 *   free_pages    : int32 [n_free] page ids to hand out, in this order (input;
 *                   may be NULL when n_free is 0)
 *   table         : int32 [batch][max_pages] (in and out: the entries for the
 *                   pages that the fresh tokens open are written, -1 where the
 *                   free pages ran out; all others are left as they are)
 *   parents       : int32 [tokens] or NULL.  With parents, sequence b's fresh
 *                   tokens are the nodes of a draft tree: parents[starts[b]+i]
 *                   is the parent's index j < i in the same sequence, or -1 for a
 *                   node that follows the last cached token; fresh <=
 *                   Q8_TREE_MAX_NODES.  Without, they are a chain.
 *   tokens        : capacity of the per-token arrays (tokens >= the sum of
 *                   fresh; a larger one is for graphs of a fixed size)
 *   starts        : int32 [batch + 1] (output) exclusive sums of fresh
 *   slots         : int32 [tokens] (output) page * page_size + offset of each
 *                   fresh token; -1 where the free pages ran out, and for
 *                   every row behind the last sequence
 *   positions     : int32 [tokens] (output): cached + the node's depth (its
 *                   place in the text); rows behind the last sequence are left
 *   masks         : int64 [tokens] (output, required with parents and NULL
 *                   without): bit j set when node j is the node itself or one of
 *                   its ancestors; rows behind the last sequence are left
 *   needed        : int32 [1] (output) pages this step opens.  Pages are
 *                   handed out by sequence, then by position; needed > n_free
 *                   says that the tokens from the first missing page on have
 *                   slot -1: run the call again, with the same held, once there
 *                   are pages enough (or with fewer sequences).
 *   held_out      : int32 [batch] (output) pages each row needs now, or NULL.
 *                   With needed <= n_free it has them: the next step's `held`.
 *                   Else it counts missing ones, whose entries of -1 are a row's
 *                   last: a row has held_out less those.  With held_out as `held`
 *                   all the same, they are reported (Q8_ERR_DATA) and their
 *                   tokens get slot -1.
 * Sequence b opens pages held .. ceil((cached+fresh)/page_size) - 1.  Running
 * the call again on the same inputs writes the same.
 * Q8_ERR_DATA: a negative length, fewer pages held than cached tokens need, a page id outside [0, n_pages), a table
 * narrower than cached + fresh, more fresh tokens than `tokens` or than
 * Q8_TREE_MAX_NODES with parents, a parent outside [-1, i).  A sequence whose
 * lengths, held pages or row width are wrong gets slots of -1 and masks of 0.
 * One with a wrong parent gets masks of 0 (its nodes see the cached tokens only)
 * and keeps its slots.  A page id out of range costs the slots in that page;
 * fresh tokens past `tokens` have no place in the per-token arrays.
 * Q8_ERR_ARG: batch outside 1..Q8_KV_MAX_BATCH, tokens < 1, page_size not a
 * positive multiple of 16, n_pages * page_size >= 2^31, masks without parents,
 * an output that overlaps an input or another output (held_out in held's
 * place: other CTAs still read held when the first ones write).
 */
Q8_API int q8_kv_plan(const int32_t *cached, const int32_t *fresh, int64_t batch, const int32_t *held,
                      const int32_t *free_pages, int64_t n_free, int32_t *table, int64_t max_pages,
                      int64_t page_size, int64_t n_pages, const int32_t *parents, int64_t tokens,
                      int32_t *starts, int32_t *slots, int32_t *positions, int64_t *masks,
                      int32_t *needed, int32_t *held_out, void *stream);

/*
 * q8_kv_append -- write the k and v rows of a step's tokens into the cache.
 *   cache, layer : cache descriptor (read during the call) and the layer
 *   k, v         : f32 [tokens][kv_heads * head_dim] (inputs, as the k and v
 *                  projections write them)
 *   slots        : int32 [tokens] (q8_kv_plan's); a token with a negative slot
 *                  is skipped, one with a slot past the cache too
 *                  (Q8_ERR_DATA).  Slots are distinct.
 * Q8_KV_F16: each value rounded to f16 (nearest even; past 65504 to infinity).
 * Q8_KV_INT8: per (token, head) row d = amax/127 in f32, code = rint(x * (1/d))
 * clamped to +-127, as a q8_0 block of head_dim values but with its scale kept
 * in f32.  One scale per row, not per 32 values: in the attention a k row's
 * scale multiplies a score and a v row's scale a softmax weight, so the codes
 * enter the tensor core as they are.  A row that holds a NaN or an infinity
 * gets a scale that is one.  tokens * kv_heads < 2^29.
 */
Q8_API int q8_kv_append(const q8_kv_cache *cache, int64_t layer, const float *k, const float *v,
                        const int32_t *slots, int64_t tokens, void *stream);

/*
 * q8_tree_attention -- attention of the fresh tokens over their sequences:
 *     y[t][h] = sum_j softmax_j(scale * q[t][h] . k[j]) v[j]
 * over the tokens j of t's sequence that t can see: every cached one, and of
 * the fresh ones (already appended) those whose bit is set in masks[t], or,
 * when masks is NULL, those not after t.  Query head h reads key/value head
 * h / (heads / kv_heads).  A row that sees nothing gives 0.
 *   q        : f32 [tokens][heads * head_dim] (input)
 *   heads    : a multiple of kv_heads, at most 64 query heads per key/value head
 *   scale    : f32, usually 1/sqrt(head_dim); finite, and so is 1.45 * scale
 *   table, max_pages, cached, starts, batch : as q8_kv_plan wrote them
 *   masks    : int64 [tokens] or NULL
 *   tokens   : rows of q and y (rows at and past starts[batch] are neither read
 *              nor written)
 *   max_fresh, max_len : host bounds: the most fresh tokens of a sequence
 *              (<= tokens; <= Q8_TREE_MAX_NODES with masks) and the most
 *              cached + fresh.  A sequence past a bound is skipped (Q8_ERR_DATA).
 *              max_fresh * heads / kv_heads decides how many rows a unit has (8,
 *              16 or 128) for all sequences of the call, so with an int8 cache
 *              give single tokens and prompt chunks calls of their own: 60
 *              tokens over up to 8191 keys and a chunk of 512 behind 2048 take
 *              272 us in one call, 152 in two (f16: 152 and 160).
 *   y        : f32 [tokens][heads * head_dim] (output), or NULL
 *   qs, ds   : q8_0 plane of y (rows at least `tokens`; rows past the last
 *              fresh one are not written), or both NULL.  Exactly the encoding
 *              of the f32 values y holds or would hold: the input of the o
 *              projection, as rmsnorm_quant and swiglu_quant produce theirs.
 *   workspace, workspace_bytes : device scratch of at least
 *              q8_tree_attention_workspace_bytes(...) bytes, 16-byte aligned;
 *              contents ignored on entry.  Two calls, or two captured graphs,
 *              may share one only if they are ordered on one stream.  NULL
 *              and 0 where q8_tree_attention_needs_workspace(...) is 0 for the
 *              call's heads, batch, max_fresh and max_len (a few rows over short
 *              contexts, which join in shared memory).
 * Precision: q enters the tensor cores as the sum of two f16 parts of its row
 * scaled by a power of two (22 bits of the row's largest value), softmax
 * weights likewise (int8: the weight times its value's scale, against the
 * largest scale the row sees), keys and values exactly as the cache holds them.
 * Statistics are f32, exponentials ex2.approx (2^-22), the quotient a product
 * with the rounded reciprocal.  Products accumulate in the tensor core's f32,
 * which rounds towards zero: about 1e-7 of the sum is lost per accumulation, and
 * at most 64 follow one another before a sum rounded to nearest, so y can lie up
 * to 6e-6 of sum p|v| nearer to zero where the values have one sign.  Against 64
 * bits, as a norm over a call, at most 1.6e-6 was measured (2.3e-6 with plain f32
 * products; over 262139 keys 1.4e-6 and 1.1e-6).  Results are run-to-run
 * identical.
 * A token that a row cannot see never enters its result, whatever it holds.  A
 * NaN or an infinity in a row's q makes the row NaN; one in a value that the
 * row sees makes what it enters non-finite.  An infinite f16 key may make the
 * rows that see it NaN also where its score would be -inf and its weight 0: q's
 * two parts may differ in sign.
 * Q8_ERR_ARG: a NULL pointer, layer or size out of range, neither y nor a
 * plane, one of qs and ds alone, a short workspace where one is needed, a scale
 * that is not finite.
 */
Q8_API size_t q8_tree_attention_workspace_bytes(const q8_kv_cache *cache, int64_t heads, int64_t max_fresh);
Q8_API int q8_tree_attention_needs_workspace(const q8_kv_cache *cache, int64_t heads, int64_t batch, int64_t max_fresh,
                                             int64_t max_len);
Q8_API int q8_tree_attention(const q8_kv_cache *cache, int64_t layer, const float *q, int64_t heads, float scale,
                             const int32_t *table, int64_t max_pages, const int32_t *cached, const int32_t *starts,
                             int64_t batch, const int64_t *masks, int64_t tokens, int64_t max_fresh,
                             int64_t max_len, float *y, int8_t *qs, uint32_t *ds, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * q8_kv_accept -- keep the verified path of each sequence's draft tree: its
 * tokens' k and v, in every layer, move to the slots right behind the cached
 * tokens, in the order of the path.
 *   table, max_pages, cached, fresh, batch : as for the step (inputs)
 *   paths    : int32 [batch][width] indices of accepted fresh tokens, strictly
 *              increasing in each row's first counts[b] entries (a path from the
 *              root through a tree is)
 *   counts   : int32 [batch], 0 .. min(width, fresh)
 *   lens     : int32 [batch] (output) cached + counts: the next step's cached
 * width 1..Q8_TREE_MAX_NODES.  k/v of token cached + paths[b][j] are copied to
 * token cached + j; other slots are left.  The pages behind the new length stay
 * in the table: give the next q8_kv_plan the step's held_out as `held`, and it
 * does not open them again.  A sequence with a bad path, count or page is left
 * as it is with lens = cached (Q8_ERR_DATA).  lens overlaps no input
 * (Q8_ERR_ARG): the layers read cached while it is written.
 */
Q8_API int q8_kv_accept(const q8_kv_cache *cache, const int32_t *table, int64_t max_pages, const int32_t *cached,
                        const int32_t *fresh, int64_t batch, const int32_t *paths, const int32_t *counts,
                        int64_t width, int32_t *lens, void *stream);

/*
 * ---------------------------------------------------------------------------
 * A mixture-of-experts block: each token's activation meets the matrices of a
 * few experts that its router logits choose on the device.  A step is
 *     router logits (any projection) -> q8_moe_route
 *     -> q8_0_experts_gate_up -> q8_0_experts_gemm (down)
 *     -> rmsnorm_residual_quant (the weighted sum, both norms, the next plane).
 *
 * A (token, expert) pair has number p = token * top_k + j, j < top_k.  Sorted by
 * expert, and by p within one, the pairs are the rows 0 .. offsets[experts] - 1
 * of the products: those of expert e are offsets[e] .. offsets[e + 1] - 1.  All
 * of this is device data, so one captured graph serves steps of any routing.
 * The kernels check each value before it becomes an address, and q8_check
 * reports Q8_ERR_DATA: an expert whose offsets are out of range or fall has no
 * rows, and with offsets that fall the rows of the others are undefined; a row
 * whose pair is out of range is left as it was.  So are rows that no expert has:
 * those before offsets[0] too, so that offsets + e0 and the matrices from expert
 * e0 on run a part of the experts.  Workspaces: two
 * calls, or two captured graphs, may share one only if they are ordered on one
 * stream; contents are ignored on entry.  Outputs overlap neither inputs nor
 * one another (Q8_ERR_ARG).
 * ---------------------------------------------------------------------------
 */
#define Q8_MAX_EXPERTS 1024
#define Q8_MAX_TOP_K   16
#define Q8_EXPERTS_MAX_N (1 << 22)   /* rows of an expert's matrix */
#define Q8_EXPERTS_MAX_K (1 << 20)   /* its columns */
#define Q8_ROUTE_CHOSEN 1   /* weights: softmax over the chosen experts */
#define Q8_ROUTE_ALL    2   /* weights: softmax over all experts */

/*
 * q8_moe_route -- the experts of each token, their weights, and the pairs
 * sorted by expert.
 *   logits : f32 [tokens][experts] (input)
 *   mode, scale : weight_j = scale * exp(l_j - max) / sum, the sum over the
 *            chosen experts (Q8_ROUTE_CHOSEN) or over all (Q8_ROUTE_ALL)
 *   valid  : int32 [1] (input) tokens that count, 0 .. tokens (Q8_ERR_DATA
 *            otherwise, and the nearest is taken), or NULL for all; the others,
 *            which fill up a graph's capacity, get no expert
 *   ids    : int32 [tokens][top_k] (output) experts by falling logit, of equal
 *            logits (+0 and -0 are) the lower expert first.  A logit that is
 *            -inf or NaN is never chosen: a token with too few others has -1 in
 *            the last places.
 *   weights: f32 [tokens][top_k] (output), 0 where ids is -1.  Logits of +inf
 *            share the weight equally.
 *   offsets: int32 [experts + 1] (output) first sorted row of each expert, and
 *            the number of pairs with an expert
 *   rows   : int32 [tokens * top_k] (output) pair of each sorted row; -1 behind
 *            the last
 *   places : int32 [tokens][top_k] (output) sorted row of each pair, -1 without
 *   workspace, workspace_bytes : device scratch of at least
 *            q8_moe_route_workspace_bytes(tokens, experts, top_k) bytes; NULL
 *            and 0 where that is 0 (few tokens).
 * experts 1..Q8_MAX_EXPERTS, top_k 1..Q8_MAX_TOP_K and <= experts, tokens >= 1,
 * tokens * top_k < 2^31, scale finite (Q8_ERR_ARG).  Results are run-to-run
 * identical.
 */
Q8_API size_t q8_moe_route_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k);
Q8_API int q8_moe_route(const float *logits, int64_t tokens, int64_t experts, int64_t top_k, int mode, float scale,
                        const int32_t *valid, int32_t *ids, float *weights, int32_t *offsets, int32_t *rows,
                        int32_t *places, void *workspace, size_t workspace_bytes, void *stream);

/*
 * q8_0_experts_gemm -- Y[r][i] = sum_b d_w(e,i,b) * d_a(s,b) * isum for the
 * sorted rows r of every expert e, s the plane row of r: the formula of
 * q8_0_gemm with the matrix chosen per row.
 *   w      : Q8_0 blocks [experts][n][k/32] (input)
 *   qs, ds, plane_rows : plane with plane_rows rows (input)
 *   offsets: int32 [experts + 1] (input, q8_moe_route's)
 *   rows   : int32 [pairs] (input, q8_moe_route's): row r reads plane row
 *            rows[r] / top_k; or NULL: it reads plane row r (an activation that
 *            is in sorted order already)
 *   pairs  : capacity of rows and y (>= offsets[experts])
 *   y      : f32 [pairs][n] (output); rows behind offsets[experts] are left
 *   workspace, workspace_bytes : at least q8_0_experts_gemm_workspace_bytes(...)
 *            bytes of device scratch; NULL and 0 where that is 0
 * k % 32 == 0, any n >= 1.  The integer dot product of a block is exact, the
 * scale of a block is rounded once and blocks are added in f32; results are
 * run-to-run identical.
 */
Q8_API size_t q8_0_experts_gemm_workspace_bytes(int64_t experts, int64_t n, int64_t k, int64_t plane_rows,
                                                int64_t top_k, int64_t pairs);
Q8_API int q8_0_experts_gemm(const void *w, int64_t experts, int64_t n, int64_t k, const int8_t *qs, const uint32_t *ds,
                             int64_t plane_rows, const int32_t *offsets, const int32_t *rows, int64_t top_k,
                             int64_t pairs, float *y, void *workspace, size_t workspace_bytes, void *stream);

/*
 * q8_0_experts_gate_up -- the gate and up products of the sorted rows and the
 * plane of silu(gate) * up, which is the input of the down product (rows NULL).
 *   w_gate, w_up : Q8_0 blocks [experts][nf][k/32] each (inputs)
 *   qs, ds, plane_rows, offsets, rows, top_k, pairs : as for q8_0_experts_gemm
 *   qs_out, ds_out : int8 [pairs][nf], uint32 [pairs][nf/32] (outputs): the
 *            plane's rows in sorted order; rows behind offsets[experts] are left
 * nf % 32 == 0.  SwiGLU and its encoding are those of swiglu_quant on the two
 * products.
 */
Q8_API size_t q8_0_experts_gate_up_workspace_bytes(int64_t experts, int64_t nf, int64_t k, int64_t plane_rows,
                                                   int64_t top_k, int64_t pairs);
Q8_API int q8_0_experts_gate_up(const void *w_gate, const void *w_up, int64_t experts, int64_t nf, int64_t k,
                                const int8_t *qs, const uint32_t *ds, int64_t plane_rows, const int32_t *offsets,
                                const int32_t *rows, int64_t top_k, int64_t pairs, int8_t *qs_out, uint32_t *ds_out,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * rmsnorm_residual_quant -- the end of a block and the start of the next in one
 * pass over the rows:
 *     b' = b + sum_j weights[t][j] * expert_rows[places[t][j]]   (either part may be absent)
 *     p  = (b' * rsqrt(mean(b'^2) + eps_post)) * w_post          (b' itself without w_post)
 *     h  = residual_scale * x + gate * p                         (gate 1 without)
 *     y  = (h * rsqrt(mean(h^2) + eps)) * w, and its q8_0 plane.
 *   x      : f32 [rows][d] (input) the residual stream
 *   b      : f32 [rows][d] (input) a dense block's output, or NULL
 *   expert_rows, expert_row_count : f32 [expert_row_count][d] (input,
 *            q8_0_experts_gemm's y), or NULL with top_k 0
 *   places, weights : [rows][top_k] (inputs, q8_moe_route's), or NULL with top_k
 *            0.  A place of -1 adds nothing; one out of range neither
 *            (Q8_ERR_DATA).
 *   w_post : f32 [d], or NULL       eps_post : read with w_post only
 *   gate   : f32 [gate_rows][d], gate_rows 1 or rows, or NULL
 *   w      : f32 [d]; NULL when neither y nor a plane is written
 *   h      : f32 [rows][d] (output), x itself allowed; or NULL
 *   y      : f32 [rows][d] (output), or NULL
 *   qs, ds, rows_pad : plane of y (output; rows rows .. rows_pad - 1 are zeros),
 *            or NULL both; exactly the encoding of the f32 values y holds or
 *            would hold
 * d % 32 == 0, d <= 32768, rows >= 0, rows_pad >= max(rows, 1); at least one
 * output; residual_scale finite, eps >= 0.  The sums run over j in order, b
 * first; each mean is an f32 sum in a fixed order.
 */
Q8_API int rmsnorm_residual_quant(const float *x, float residual_scale, const float *b, const float *expert_rows,
                                  int64_t expert_row_count, const int32_t *places, const float *weights, int64_t top_k,
                                  const float *w_post, float eps_post, const float *gate, int64_t gate_rows,
                                  const float *w, float eps, float *h, float *y, int64_t rows, int64_t d, int8_t *qs,
                                  uint32_t *ds, int64_t rows_pad, void *stream);

/*
 * q8_check -- synchronise `stream`, then read and clear the library's device
 * error words.  Returns Q8_OK, Q8_ERR_DEVICE_TIMEOUT if a bounded on-device
 * wait ran out since the last check (the affected outputs are undefined; also
 * when there is the next to report), Q8_ERR_DATA if the key/value cache's or the
 * experts' calls met a value out of range, or Q8_ERR_CUDA if the synchronisation itself failed.
 */
Q8_API int q8_check(void *stream);

/* Number of SMs of the current device (0 on error); used by the host-side
 * dispatch and exported for tests. */
Q8_API int q8_num_sms(void);

#ifdef __cplusplus
}
#endif
#endif /* Q8PROJ_H */
