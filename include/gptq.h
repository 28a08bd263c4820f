/*
 * gptq.h -- C ABI of a GB300 (sm_103a) library for GPTQ's per-layer second-order
 * weight quantization.
 *
 * The operation (three web pages on GPTQ: "GPTQ › Mathematical Details of the Update";
 * "tm_gptq_math"; "GPTQ Hessian", excerpt of "GPTQ: Block Structure in Quantization"):
 * for one linear layer with weights W [d_out, d_in] and calibration inputs X, find a
 * few-bit W_hat whose outputs on X stay close to W's, one row at a time, all rows sharing
 * the Hessian H = 2 X X^T of the per-row quadratic error.  The path is split into the
 * three calls below, in the pages' order:
 *
 *   gptq_hessian_accumulate   X -> H          ("tm_gptq_math", "Why it is second-order:
 *                                               the Hessian")
 *   gptq_prepare              H -> U          ("tm_gptq_math", "The Cholesky trick for the
 *                                               inverse Hessian"; "GPTQ Hessian")
 *   gptq_quantize_layer       W, U -> codes   ("tm_gptq_math", "Greedy quantization with
 *                                               error compensation" and "GPTQ's speedups:
 *                                               fixed order and lazy batches"; "GPTQ Hessian")
 *
 * Conventions shared by every call
 *   - All matrices are row-major.  X is token-major [n_tok, d_in] (row t = input x_t, so
 *     the pages' X of shape [d_in, N] is X^T here).  W is [d_out, d_in].
 *   - Every pointer is a DEVICE pointer on the current CUDA device unless marked "host".
 *     The library never allocates, frees or keeps device memory beyond a call; the caller
 *     owns every buffer.  Scratch memory is a caller-supplied workspace whose size the
 *     *_workspace_bytes functions give; it must be 256-byte aligned.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Kernels are
 *     enqueued on it; calls return once work is enqueued unless stated otherwise.
 *   - Argument errors are reported synchronously, before anything is enqueued.  A failed
 *     kernel launch returns GPTQ_ERR_CUDA.
 *   - The calls are thread-compatible: concurrent calls must use distinct outputs and
 *     workspaces.
 */
#ifndef GPTQ_GB300_H
#define GPTQ_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GPTQ_ABI_VERSION 1

typedef struct CUstream_st *gptq_stream_t; /* identical to cudaStream_t */

typedef enum gptq_status {
  GPTQ_OK = 0,
  GPTQ_ERR_INVALID_ARG = 1,  /* bad size, dtype, bit width, block, null or misaligned ptr */
  GPTQ_ERR_NOT_PD = 2,       /* damped Hessian not positive definite (gptq_prepare)       */
  GPTQ_ERR_NONFINITE = 3,    /* NaN/Inf found in an input                                 */
  GPTQ_ERR_TIMEOUT = 4,      /* a bounded device-side wait gave up                        */
  GPTQ_ERR_CUDA = 5,         /* a CUDA runtime call or kernel launch failed               */
  GPTQ_ERR_UNSUPPORTED = 6,  /* valid request this library does not implement             */
  GPTQ_ERR_WORKSPACE = 7     /* workspace missing, too small or not 256-byte aligned      */
} gptq_status;

typedef enum gptq_dtype { GPTQ_F16 = 0, GPTQ_BF16 = 1, GPTQ_F32 = 2 } gptq_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char *gptq_status_str(int status);

/* GPTQ_ABI_VERSION of the loaded library. */
int gptq_abi_version(void);

/* Number of CUDA kernels this library has launched in this process (all threads). */
unsigned long long gptq_kernel_launches(void);

/*
 * gptq_hessian_accumulate: H = (accumulate ? H : 0) + 2 * X^T X.
 *
 * Source: "tm_gptq_math", "Why it is second-order: the Hessian" -- the per-row output
 * error is a quadratic in the row's weights whose constant Hessian is twice the Gram
 * matrix of the inputs; "GPTQ Hessian" -- every row of the layer shares it.  Calling this
 * once per token chunk with accumulate=1 after the first accumulates the Hessian of the
 * whole calibration set while only one chunk of X is resident.
 *
 *   X          [n_tok, ldx] elements of type `xdtype`, first d_in columns used; 16-byte
 *              aligned, ldx * sizeof(elem) a multiple of 16 bytes.
 *   xdtype     GPTQ_F16 / GPTQ_BF16 (tensor-core path, fp32 accumulation) or GPTQ_F32.
 *   n_tok      >= 0 tokens (0 leaves H as is, or zero when accumulate=0).
 *   d_in       >= 1 input channels.
 *   H          [d_in, d_in] fp32, both triangles written.  With accumulate=1 the lower
 *              triangle of the existing H is read and the result is written symmetric.
 * Asynchronous.  Errors: INVALID_ARG, CUDA.
 */
gptq_status gptq_hessian_accumulate(const void *X, int xdtype, int64_t n_tok, int64_t d_in,
                                    int64_t ldx, float *H, int accumulate,
                                    gptq_stream_t stream);

/*
 * gptq_hessian_host_workspace_bytes: device staging workspace that
 * gptq_hessian_accumulate_host needs for inputs of d_in channels streamed in chunks of
 * chunk_tok tokens (0 = the default chunk: about 64 MiB of X, a multiple of 512 tokens, and
 * at least 8192 tokens, or 32768 from d_in = 16384 on, since every chunk's products read and
 * write all of H).
 * Returns 0 for an unknown dtype, d_in < 1 or chunk_tok < 0.
 */
size_t gptq_hessian_host_workspace_bytes(int xdtype, int64_t d_in, int64_t chunk_tok);

/*
 * gptq_hessian_accumulate_host: gptq_hessian_accumulate with X in HOST memory.
 *
 * Source: as gptq_hessian_accumulate ("tm_gptq_math", "Why it is second-order: the
 * Hessian"); the pages accumulate the Gram matrix over the calibration set, which is what
 * the chunks below do.  The pages have no counterpart to the host staging itself: it
 * exists so that the calibration activations need not be resident on the GPU, and so that
 * their transfer overlaps the Gram products.
 *
 * X is copied to the device in chunks of chunk_tok tokens through two staging buffers in
 * `ws`; the copy of chunk c + 1 runs on a copy stream this library keeps per device while
 * chunk c is accumulated into H on `stream`.  Chunks are accumulated in token order, each
 * exactly as one gptq_hessian_accumulate call over that chunk would (so the fp32 sums are
 * grouped by chunk; the result can differ in the last bits from one call over all tokens).
 *
 *   X_host     HOST [n_tok, ldx] elements of xdtype, first d_in columns used.  Page-locked
 *              memory (cudaHostAlloc / cudaHostRegister) lets the copies overlap; pageable
 *              memory gives the same result, but each copy then blocks the calling thread.
 *              Must stay valid and unchanged until the work on `stream` has completed.
 *   xdtype     GPTQ_F16, GPTQ_BF16 or GPTQ_F32;  d_in * sizeof(elem) a multiple of 16 bytes.
 *   n_tok      >= 0;  ldx >= d_in (host rows may be strided; no alignment needed).
 *   H          as gptq_hessian_accumulate (DEVICE, 16-byte aligned); `accumulate` applies
 *              to the first chunk, later chunks always accumulate.
 *   chunk_tok  tokens per chunk (0 = default); the same value as in the size query.
 *   ws         DEVICE workspace, 256-byte aligned, of ws_bytes >=
 *              gptq_hessian_host_workspace_bytes(xdtype, d_in, chunk_tok).
 * Returns once everything is enqueued (for page-locked X); every copy and product is
 * ordered before later work on `stream`, and the copies start only after earlier work on
 * `stream` (which may still use `ws`) has finished.  Calls from several host threads are
 * serialized while they enqueue.  Errors: INVALID_ARG, WORKSPACE, CUDA.
 */
gptq_status gptq_hessian_accumulate_host(const void *X_host, int xdtype, int64_t n_tok,
                                         int64_t d_in, int64_t ldx, float *H, int accumulate,
                                         int64_t chunk_tok, void *ws, size_t ws_bytes,
                                         gptq_stream_t stream);

/*
 * gptq_prepare_workspace_bytes: workspace size gptq_prepare needs for this d_in.
 */
size_t gptq_prepare_workspace_bytes(int64_t d_in);

/*
 * gptq_prepare: dead columns, damping and the inverse-Hessian Cholesky factor.
 *
 * Source: "tm_gptq_math", "The Cholesky trick for the inverse Hessian" -- channels with a
 * zero Hessian diagonal are skipped, the diagonal is damped by lambda = damp * mean(diag)
 * (about 1 %), and one Cholesky factorization of the inverse supplies every row the
 * fixed-order sweep needs; "GPTQ Hessian" -- U is the upper-triangular factor with
 * H^-1 = U^T U; "GPTQ › Mathematical Details of the Update" writes it as L = U^T.
 *
 * Steps: dead = {i : H_ii == 0}; H_ii = 1 for dead i; lambda = damp * mean(diag H) (after
 * that fix, over all d_in entries); H += lambda I; U = upper Cholesky factor of H^-1.
 * U is computed as the inverse of the reversed-order ("UL") Cholesky factor R of H
 * (H = R R^T, R upper), which is the same matrix.
 *
 *   H          [d_in, d_in] fp32 symmetric, CONSUMED: overwritten as scratch.  Only the
 *              upper triangle and the diagonal are read (the lower triangle may hold anything).
 *   d_in       >= 1.
 *   damp       >= 0 relative damping (0.01 for the pages' 1 %).
 *   U          [d_in, d_in] fp32 out, upper triangular (lower triangle written as 0).
 *   dead_mask  [d_in] uint8 out (1 = dead), may be NULL.
 *   n_dead     HOST int32 out, may be NULL.
 *   ws         workspace of ws_bytes >= gptq_prepare_workspace_bytes(d_in).
 * SYNCHRONIZES `stream` before returning.  Errors: INVALID_ARG, WORKSPACE, NOT_PD (a
 * pivot <= 0: U is then undefined), NONFINITE (NaN/Inf in the part of H read), CUDA.
 *
 * Repeatability: the factorization runs on several streams of this library that add into
 * shared blocks of the workspace in an order that is not fixed, so two calls on the same
 * H can give U's that differ in their last bits (relative row differences of order 1e-6).
 * A sweep on either gives the same codes except where a weight sits within rounding noise
 * of a grid boundary (the two codes are then adjacent).
 */
gptq_status gptq_prepare(float *H, int64_t d_in, float damp, float *U, uint8_t *dead_mask,
                         int32_t *n_dead, void *ws, size_t ws_bytes, gptq_stream_t stream);

/*
 * gptq_quantize_workspace_bytes: workspace size gptq_quantize_layer needs.
 */
size_t gptq_quantize_workspace_bytes(int64_t d_out, int64_t d_in, int bits, int block);

/*
 * gptq_quantize_layer: the GPTQ column sweep of one layer.
 *
 * Source: "tm_gptq_math", "Greedy quantization with error compensation" (quantize one
 * weight, move the still-free weights by the optimal correction), "GPTQ's speedups:
 * fixed order and lazy batches" (one left-to-right column order for all rows; blocks of
 * `block` columns, corrections inside the block applied at once, corrections of later
 * columns deferred to one product per block); "GPTQ Hessian" (row j of U supplies the
 * correction of column j); "GPTQ › Mathematical Details of the Update" (O(d_in) work per
 * column once the factor exists).
 *
 * Grid (the pages define none; this library's reading): per output row i, asymmetric
 * min-max over W's row as given, with 0 inside the range:
 *   x_min = min(0, min_j W_ij), x_max = max(0, max_j W_ij),
 *   scale_i = (x_max - x_min) / (2^bits - 1)  (1 if that is 0),  zero_i = rint(-x_min/scale_i)
 * in fp32.  Dead columns (dead_mask) are set to 0 before the sweep.  For each column j in
 * order, with w the current fp32 working value:
 *   code = clamp(rint(w / scale) + zero, 0, 2^bits - 1)      (IEEE division, ties to even)
 *   q = scale * (code - zero);  e = (w - q) / U_jj
 *   w_k -= e * U_jk for every later column k (inside the block at once, later columns
 *   through the deferred block product).
 *
 *   W          [d_out, ldw] of type `wdtype` (GPTQ_BF16, GPTQ_F16 or GPTQ_F32), not modified.
 *   d_out      >= 1 rows;  d_in >= 1 columns;  ldw >= d_in.
 *   U          [d_in, d_in] fp32 upper factor from gptq_prepare (only the upper triangle
 *              is read).
 *   dead_mask  [d_in] uint8 (nonzero = dead) or NULL.
 *   bits       2, 3, 4 or 8.
 *   block      lazy-batch width B: 1 <= B <= 128 (128 is the pages' value).
 *   qpacked    [d_out, ceil(d_in/32) * bits] uint32 out: row-wise little-endian
 *              bitstream, the code of column c in bits [c*bits, (c+1)*bits) of its row
 *              (bit b of the stream = bit b%32 of word b/32); padding bits are 0.
 *   scale      [d_out] fp32 out;  zero: [d_out] int32 out.
 *   W_hat      [d_out, d_in] fp32 out (scale * (code - zero)), or NULL.
 *   ws         workspace of ws_bytes >= gptq_quantize_workspace_bytes(d_out, d_in, bits,
 *              block); its contents need no initialisation.
 * Asynchronous.  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.  Non-finite weights
 * are flagged in the workspace; read the flag with gptq_workspace_status.
 */
gptq_status gptq_quantize_layer(const void *W, int wdtype, int64_t d_out, int64_t d_in,
                                int64_t ldw, const float *U, const uint8_t *dead_mask,
                                int bits, int block, uint32_t *qpacked, float *scale,
                                int32_t *zero, float *W_hat, void *ws, size_t ws_bytes,
                                gptq_stream_t stream);

/*
 * GPTQ_MAX_SHARED_LAYERS: most layers one gptq_quantize_layers_shared call takes.
 */
#define GPTQ_MAX_SHARED_LAYERS 64

/*
 * gptq_quantize_shared_workspace_bytes: workspace size gptq_quantize_layers_shared needs
 * for n_layers layers of d_out[i] rows (HOST array) and d_in columns.  0 for bad arguments.
 */
size_t gptq_quantize_shared_workspace_bytes(int n_layers, const int64_t *d_out, int64_t d_in,
                                            int bits, int block);

/*
 * gptq_quantize_layers_shared: the column sweep of several layers that read the same
 * inputs, sharing one U.
 *
 * Source: "GPTQ Hessian" -- H depends on the layer inputs only and every row of W shares
 * it, and the rows are quantized independently of one another.  Layers fed by the same
 * inputs (the query, key and value projections of an attention block; the gate and up
 * projections of an MLP) therefore share H, its damping and U, and their rows can be swept
 * as one stack.  The pages have no multi-layer call; this one avoids concatenating the
 * weights on the caller's side and runs one sweep and one trailing update per block over
 * all rows.
 *
 * Each layer's outputs are exactly those of gptq_quantize_layer on that layer alone (same
 * codes, scales, zeros and W_hat, bit for bit).
 *
 *   n_layers   1 .. GPTQ_MAX_SHARED_LAYERS.
 *   W, wdtype, d_out, ldw, qpacked, scale, zero
 *              HOST arrays of n_layers entries; entry i describes layer i exactly as the
 *              same-named argument of gptq_quantize_layer (the pointers are DEVICE pointers).
 *   W_hat      HOST array of n_layers DEVICE pointers (entries may be NULL), or NULL.
 *   d_in, U, dead_mask, bits, block: shared by all layers, as in gptq_quantize_layer.
 *   ws         workspace of ws_bytes >= gptq_quantize_shared_workspace_bytes(...).
 * The host arrays are read during the call only.  Asynchronous.  Errors: INVALID_ARG,
 * WORKSPACE, UNSUPPORTED, CUDA; non-finite weights are flagged in the workspace
 * (gptq_workspace_status).
 */
gptq_status gptq_quantize_layers_shared(int n_layers, const void *const *W, const int *wdtype,
                                        const int64_t *d_out, const int64_t *ldw, int64_t d_in,
                                        const float *U, const uint8_t *dead_mask, int bits,
                                        int block, uint32_t *const *qpacked,
                                        float *const *scale, int32_t *const *zero,
                                        float *const *W_hat, void *ws, size_t ws_bytes,
                                        gptq_stream_t stream);

/*
 * gptq_recon_error_workspace_bytes: workspace size gptq_recon_error needs.  0 for bad
 * arguments.
 */
size_t gptq_recon_error_workspace_bytes(int xdtype, int64_t d_out, int64_t d_in,
                                        int64_t n_tok);

/*
 * gptq_recon_error: per-row output error of a quantized layer on its inputs,
 *   err[i] = sum_t ( (W_i - W_hat_i) . x_t )^2 ,   W_hat = scale * (code - zero),
 * so that sum_i err[i] = ||W X^T - W_hat X^T||_F^2 with X token-major.
 *
 * Source: "tm_gptq_math", "The reconstruction objective, written out" -- GPTQ minimizes
 * this squared output error, one row at a time, over the calibration inputs.  The codes are
 * read from the packed form gptq_quantize_layer writes, so this is the consumer of the
 * quantized layer; it evaluates the objective on X directly rather than through H.
 *
 *   X          [n_tok, ldx] of xdtype: GPTQ_F16 / GPTQ_BF16 (tensor cores: W - W_hat is
 *              rounded to the same type, fp32 accumulation) or GPTQ_F32 (CUDA cores);
 *              16-byte aligned, ldx * sizeof(elem) a multiple of 16 bytes.
 *   W          [d_out, ldw] of wdtype, the layer's original weights.
 *   qpacked, bits, scale, zero
 *              as written by gptq_quantize_layer for this W (packed rows of
 *              ceil(d_in/32) * bits words).
 *   err        [d_out] fp32 out.
 *   ws         workspace of ws_bytes >= gptq_recon_error_workspace_bytes(...).
 * The row sums are combined in a fixed order: repeated calls give identical results.
 * Asynchronous.  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.
 */
gptq_status gptq_recon_error(const void *X, int xdtype, int64_t n_tok, int64_t d_in,
                             int64_t ldx, const void *W, int wdtype, int64_t d_out, int64_t ldw,
                             const uint32_t *qpacked, int bits, const float *scale,
                             const int32_t *zero, float *err, void *ws, size_t ws_bytes,
                             gptq_stream_t stream);

/*
 * GPTQ_OBQ_MAX_D_IN: widest layer gptq_quantize_obq takes (its per-row inverse Hessian
 * lives in on-chip shared memory).
 */
#define GPTQ_OBQ_MAX_D_IN 128

/*
 * gptq_quantize_obq_workspace_bytes: workspace size gptq_quantize_obq needs.  0 for bad
 * arguments.
 */
size_t gptq_quantize_obq_workspace_bytes(int64_t d_out, int64_t d_in);

/*
 * gptq_quantize_obq: the greedy-order variant that GPTQ's fixed order replaces.
 *
 * Source: "tm_gptq_math", "Greedy quantization with error compensation" -- per row,
 * quantize next the free weight whose rounding raises the output error least,
 * (w_q - quant(w_q))^2 / [H_F^-1]_qq, and correct the other free weights by
 * -((w_q - quant(w_q)) / [H_F^-1]_qq) H_F^-1[:, q]; "GPTQ › Mathematical Details of the
 * Update" -- remove q from the free set by the rank-one Schur downdate of H_F^-1.  Every
 * row follows its own order, so each row carries its own H_F^-1: O(d_in^3) per row, for
 * small layers.  Costs are compared in fp32; ties go to the lowest column index.
 *
 * Same grid, dead-column handling and outputs as gptq_quantize_layer, plus:
 *   U          [d_in, d_in] fp32 upper factor from gptq_prepare (H^-1 = U^T U is formed
 *              from it).
 *   d_in       1 .. GPTQ_OBQ_MAX_D_IN (else UNSUPPORTED).
 *   order      [d_out, d_in] int32 out, or NULL: row i's columns in the order quantized.
 *   ws         workspace of ws_bytes >= gptq_quantize_obq_workspace_bytes(d_out, d_in).
 * Asynchronous.  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.
 */
gptq_status gptq_quantize_obq(const void *W, int wdtype, int64_t d_out, int64_t d_in,
                              int64_t ldw, const float *U, const uint8_t *dead_mask, int bits,
                              uint32_t *qpacked, float *scale, int32_t *zero, float *W_hat,
                              int32_t *order, void *ws, size_t ws_bytes, gptq_stream_t stream);

/*
 * GPTQ_NOALLOC_SCRATCH_BYTES: size of the fixed scratch array behind
 * gptq_quantize_layer_noalloc (32 MiB per GPU, from the first call on that GPU until the
 * process exits).  A layer fits when
 * gptq_quantize_workspace_bytes(d_out, d_in, bits, block) <= GPTQ_NOALLOC_SCRATCH_BYTES
 * (for example 1024 x 1024 at 4 bits, B = 128).
 */
#define GPTQ_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * gptq_quantize_layer_noalloc: gptq_quantize_layer for callers that cannot allocate.
 *
 * The pages have no counterpart to this call; it exists for callers that cannot call
 * cudaMalloc: code embedded in a host framework that owns all device memory and forbids
 * allocations while it runs, or code that must not cause the device-wide synchronization
 * an allocation or free can bring.  It computes exactly what gptq_quantize_layer computes,
 * with the same arguments minus the workspace: its scratch is a fixed array inside the
 * library (GPTQ_NOALLOC_SCRATCH_BYTES per GPU), and the call itself allocates nothing.
 *
 *   - Sizes: returns GPTQ_ERR_WORKSPACE, before touching the GPU, when the layer needs more
 *     scratch than GPTQ_NOALLOC_SCRATCH_BYTES; use gptq_quantize_layer with a workspace then.
 *   - First call on a device: looks up the array's device address (once per device, with
 *     that device current).  Under CUDA's default lazy module loading this look-up is also
 *     what loads the library code that holds the array, so the first call reserves the
 *     32 MiB on that device and may synchronize it: make the first call during set-up, and
 *     before any stream capture.  Only the later calls allocate nothing.
 *   - Sharing: every call on a device uses the same array, which keeps the last call's
 *     contents (each call clears what it needs).  Calls whose GPU work overlaps (e.g. on
 *     two unordered streams) race and give wrong results: keep them on one stream.
 *   - Device-side status (non-finite weights; a bounded wait that gave up, after which the
 *     outputs are undefined) is recorded in the shared array: read it with
 *     gptq_noalloc_status after the call.
 * Asynchronous.  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.
 */
gptq_status gptq_quantize_layer_noalloc(const void *W, int wdtype, int64_t d_out, int64_t d_in,
                                        int64_t ldw, const float *U, const uint8_t *dead_mask,
                                        int bits, int block, uint32_t *qpacked, float *scale,
                                        int32_t *zero, float *W_hat, gptq_stream_t stream);

/*
 * gptq_noalloc_status: synchronize `stream`, then return the device-side status the last
 * gptq_quantize_layer_noalloc on the current device recorded: GPTQ_OK, GPTQ_ERR_NONFINITE
 * (a NaN or Inf in W) or GPTQ_ERR_TIMEOUT (a bounded device wait gave up; the outputs of
 * that call are undefined).  Allocates nothing after the first gptq_quantize_layer_noalloc
 * call on the device (see there).  Errors of its own: CUDA.
 */
gptq_status gptq_noalloc_status(gptq_stream_t stream);

/*
 * gptq_workspace_status: synchronize `stream`, then return the device-side status the
 * last gptq_quantize_layer on workspace `ws` recorded (GPTQ_OK, GPTQ_ERR_NONFINITE or
 * GPTQ_ERR_TIMEOUT).  `ws` must be a workspace that call used.
 */
gptq_status gptq_workspace_status(const void *ws, gptq_stream_t stream);

/*
 * gptq_debug_hessian_lost_stage: test hook of the bounded device waits (the pages have no
 * counterpart; it exists so that the failure path of the tensor-core kernels can be tested
 * without hanging a GPU).
 *
 * Runs the fp16/bf16 tensor-core Hessian exactly as gptq_hessian_accumulate with
 * accumulate = 0 would, except that its TMA producer issues nothing for token stage
 * `lost_stage` (stages are 128 tokens): no copy and no arrival, so the MMA issuer's wait for
 * that stage can never complete.  Every wait of the launch gives up after `wait_ns`
 * nanoseconds of the GPU's global timer, records GPTQ_ERR_TIMEOUT in the status block and
 * returns; the CTA then leaves with no copy or tensor-core operation of its own in flight
 * and its tensor memory freed, so the context stays usable.
 *
 *   X, xdtype, n_tok, d_in, ldx, H
 *              as gptq_hessian_accumulate; xdtype GPTQ_F16 or GPTQ_BF16 with d_in >= 64
 *              and n_tok >= 64 (else UNSUPPORTED).  H is left undefined.
 *   lost_stage 0 <= lost_stage < ceil(n_tok / 128).
 *   wait_ns    1e3 .. 1e10: budget of every wait (the regular calls use 2 s).
 *   status_ws  DEVICE buffer of >= 256 bytes, 256-byte aligned, for the status block.
 * SYNCHRONIZES `stream` and returns the device status: GPTQ_ERR_TIMEOUT when the waits ran
 * out as designed.  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.
 */
gptq_status gptq_debug_hessian_lost_stage(const void *X, int xdtype, int64_t n_tok,
                                          int64_t d_in, int64_t ldx, float *H,
                                          int64_t lost_stage, uint64_t wait_ns, void *status_ws,
                                          gptq_stream_t stream);

/* ======================================================================================
 * 8-bit serving of quantized layers
 *
 * The pages end with the quantized layer; the calls below run a decoder on such layers with
 * 8-bit operands, and have no counterpart in the pages.
 *
 * Number format: e4m3 codes with one exponent byte E for each block of elements; an element
 * is code * 2^(E - 127).  A block whose largest finite magnitude is a has
 *   e = ceil(log2(a / 448)) limited to [-96, 120]  (-96 for a block of zeros),  E = e + 127,
 * and its codes are x * 2^-e rounded to nearest even.  An element that is not finite becomes
 * the NaN code.  A matrix [rows, d] of this format is
 *   codes  [rows, ldc] bytes, 16-byte aligned, ldc a multiple of 16 and >= d;
 *   exps   [rows or ceil(rows / 128), lde] bytes, 4-byte aligned, lde a multiple of 4 and
 *          >= ceil(d / 128): blocks of 1 x 128 (activations) or 128 x 128 (weights) elements;
 *   and optionally an fp32 factor per row (the norm's 1/rms; GPTQ's per-row step).
 * Bytes between a row's end and its pitch are neither read into a result nor written.
 * Matrices of more than 2^20 columns or 2^22 rows are refused (UNSUPPORTED).
 * ====================================================================================== */

/*
 * gptq_rmsnorm_fp8: h = X + R;  u = h * weight;  rstd = (mean(h^2) + eps)^-1/2 per row;
 * codes and exponents of u by 1 x 128 blocks.  The normalised row is rstd * u: rstd is handed
 * to gptq_fp8_matmul as the row's scale (the codes of a floating format are the same with or
 * without it).  h and u are taken in fp32 (u from the unrounded h); H is h rounded to xdtype.
 *
 *   X, R, H    [rows, d] of xdtype (F16, BF16 or F32) with row pitches ldx, ldr, ldh >= d.  R
 *              (the residual) and H may be NULL; H may be X or R itself.  Rows are read and
 *              written in the widest words (16, 8, 4 bytes) that their alignment allows.
 *   weight     [d] of wdtype: xdtype, or F32.
 *   rows >= 0, d >= 1; eps >= 0.   rstd [rows] fp32 out.
 * Asynchronous.  Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
gptq_status gptq_rmsnorm_fp8(const void *X, int xdtype, int64_t rows, int64_t d, int64_t ldx,
                             const void *R, int64_t ldr, const void *weight, int wdtype,
                             float eps, void *H, int64_t ldh, uint8_t *codes, int64_t ldc,
                             uint8_t *exps, int64_t lde, float *rstd, gptq_stream_t stream);

/*
 * gptq_fp8_quantize: X [rows, d] of xdtype to e4m3 codes and exponents, by blocks of
 * row_block x 128 elements: row_block 1 (activations) or 128 (weights).
 * Asynchronous.  Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
gptq_status gptq_fp8_quantize(const void *X, int xdtype, int64_t rows, int64_t d, int64_t ldx,
                              int row_block, uint8_t *codes, int64_t ldc, uint8_t *exps,
                              int64_t lde, gptq_stream_t stream);

/*
 * gptq_fp8_from_codes: the packed codes of gptq_quantize_layer as an e4m3 weight matrix of
 * 128 x 128 blocks: code - zero, an integer in [-15, 15] at 2, 3 and 4 bits, is an exact e4m3
 * value; every exponent is 2^0.  With gptq_quantize_layer's scale as the row factor the
 * matrix is exactly W_hat.  8-bit codes do not fit e4m3: UNSUPPORTED.
 *   qpacked, bits, zero: as written by gptq_quantize_layer for [d_out, d_in].
 * Asynchronous.  Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
gptq_status gptq_fp8_from_codes(const uint32_t *qpacked, int bits, const int32_t *zero,
                                int64_t d_out, int64_t d_in, uint8_t *codes, int64_t ldc,
                                uint8_t *exps, int64_t lde, gptq_stream_t stream);

/*
 * gptq_fp8_matmul_workspace_bytes: workspace size gptq_fp8_matmul needs.  0 for bad arguments.
 */
size_t gptq_fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k);

/*
 * gptq_fp8_matmul: out [m, n] = diag(a_scale) A W^T diag(w_scale), A [m, k] in 1 x 128 blocks
 * and W [n, k] in 128 x 128 blocks; products accumulated in fp32, rounded once to odtype.
 *
 *   a_scale    [m] fp32 or NULL (1);  w_scale: [n] fp32 or NULL (1).
 *   out        [m, ldo] of odtype (F16 or BF16), ldo >= n.
 *   m >= 0 (0: nothing is done), n >= 1, k >= 1.
 *   ws         workspace of ws_bytes >= gptq_fp8_matmul_workspace_bytes(m, n, k).
 * Repeated calls give identical results.  Asynchronous; a bounded device wait that gave up is
 * recorded in ws (gptq_workspace_status).  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.
 */
gptq_status gptq_fp8_matmul(const uint8_t *a, int64_t lda, const uint8_t *a_exps, int64_t ldae,
                            const float *a_scale, const uint8_t *w, int64_t ldw,
                            const uint8_t *w_exps, int64_t ldwe, const float *w_scale, int64_t m,
                            int64_t n, int64_t k, void *out, int odtype, int64_t ldo, void *ws,
                            size_t ws_bytes, gptq_stream_t stream);

/*
 * The 8-bit cache of keys and values: n_blocks blocks of GPTQ_KV8_BLOCK tokens,
 *   k       [n_blocks, n_kv, GPTQ_KV8_BLOCK, dim] e4m3 codes (16-byte aligned),
 *   v       [n_blocks, n_kv, dim, GPTQ_KV8_BLOCK] e4m3 codes (16-byte aligned; a channel's
 *           tokens lie together),
 *   k_exps, v_exps   [n_blocks, n_kv] exponent bytes, one for each block and head,
 * and for each sequence a row of `table` [n_seq, ld_table] int32: table[s][i] is the block that
 * holds its tokens [64 i, 64 i + 64).  An index outside [0, n_blocks) stands for tokens that are
 * not there: they are not attended to, and appends to them are dropped.
 * Limits, beyond which the calls return UNSUPPORTED: dim 64 or 128; n_seq, n_heads <= 65535;
 * n_kv <= 4096; n_new, max_blocks <= 2^20; n_blocks * n_kv < 2^31; and, for the attention,
 * n_seq * n_kv * (tiles of n_new * n_heads / n_kv rows) * max_blocks below about 2^30.
 */
#define GPTQ_KV8_BLOCK 64

/*
 * gptq_kv8_append: writes n_new tokens of each sequence at its tokens [start[s], start[s] + n_new).
 * A block's exponents are raised to what the new tokens need and the codes of the block's
 * tokens before start[s] are then re-rounded by that power of two; slots after the new tokens
 * keep their bytes.  A block that the new tokens begin takes its exponents from them alone.  A
 * token whose value is not finite somewhere is stored with NaN codes in its key: exactly the
 * rows that attend to it become NaN.
 *
 *   new_k, new_v   [n_seq, n_new, n_kv, dim] of dtype (F16, BF16 or F32), elements of a head
 *                  contiguous; k_strides, v_strides: HOST arrays of three element strides
 *                  (sequence, token, head), >= 0.
 *   dim            64 or 128 (else UNSUPPORTED).
 *   start          [n_seq] int32; tokens past max_blocks * 64 are dropped, and so is a
 *                  sequence whose start is negative.
 * No two sequences may append to one block.  Asynchronous.  Errors: INVALID_ARG, UNSUPPORTED,
 * CUDA.
 */
gptq_status gptq_kv8_append(const void *new_k, const int64_t *k_strides, const void *new_v,
                            const int64_t *v_strides, int dtype, int64_t n_seq, int64_t n_new,
                            int n_kv, int dim, uint8_t *k, uint8_t *v, uint8_t *k_exps,
                            uint8_t *v_exps, int64_t n_blocks, const int32_t *table,
                            int64_t ld_table, int64_t max_blocks, const int32_t *start,
                            gptq_stream_t stream);

/*
 * gptq_kv8_attention_workspace_bytes: workspace size gptq_kv8_attention needs.  0 for bad
 * arguments.
 */
size_t gptq_kv8_attention_workspace_bytes(int64_t n_seq, int64_t n_new, int n_heads, int n_kv,
                                          int dim, int64_t max_blocks);

/*
 * gptq_kv8_attention: out = softmax(scale * q K^T) V over the cached tokens, for the last
 * n_new tokens of each sequence (their keys and values are already in the cache).
 *
 *   q, out     [n_seq, n_new, n_heads, dim] of dtype (F16 or BF16), elements of a head
 *              contiguous; q_strides, o_strides: HOST arrays of three element strides.  Rows of
 *              q may coincide, rows of out may not overlap.
 *              Query head h reads cache head h / (n_heads / n_kv).
 *   lengths    [n_seq] int32: tokens of the sequence in the cache, the new ones included,
 *              limited to [0, 64 * max_blocks].  With causal != 0 new token t sees the tokens
 *              [0, length - n_new + t], otherwise all `length` of them.  A row that sees
 *              nothing gives zeros; one whose query is not finite gives NaN.  Bytes of the
 *              cache past `length` never matter.
 *   scale      factor of the scores (finite).
 *   Scores, their statistics and sums are fp32, of queries held to 2^-17 of their largest element
 *   or better.  Probabilities, weighted by their block's value scale, are multiplied as numbers
 *   - of 9 bits (BF16) or 12 bits (F16) where few rows share a cache head (a decoding step): a small
 *     one may be off by 2^-23 of its block's largest where that is hidden, to 2^-9, in the row's sums,
 *     and one below 2^-40 of the row's largest adds to the softmax's sum alone;
 *   - of 11 bits (fp16) in prompts: with fewer from 2^-24 of the row's largest on, and one below 2^-33
 *     adds to the softmax's sum alone.
 *   The width max_blocks of the table, not the lengths, chooses the kernel and the way that its work
 *   is dealt (and sizes ws): a table much wider than the histories in it costs short ones time.
 *   ws         workspace of ws_bytes >= gptq_kv8_attention_workspace_bytes(...).
 * Repeated calls give identical results.  Asynchronous; a bounded device wait that gave up is
 * recorded in ws (gptq_workspace_status).  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.
 */
gptq_status gptq_kv8_attention(const void *q, const int64_t *q_strides, int dtype, int64_t n_seq,
                               int64_t n_new, int n_heads, int n_kv, int dim, const uint8_t *k,
                               const uint8_t *v, const uint8_t *k_exps, const uint8_t *v_exps,
                               int64_t n_blocks, const int32_t *table, int64_t ld_table,
                               int64_t max_blocks, const int32_t *lengths, int causal,
                               float scale, void *out, const int64_t *o_strides, void *ws,
                               size_t ws_bytes, gptq_stream_t stream);

/*
 * gptq_serving_status: synchronize `stream`, then return GPTQ_ERR_TIMEOUT if a bounded device wait
 * of a gptq_fp8_matmul, gptq_kv8_attention or one of the products of feed-forward blocks on the
 * current device, on whichever stream and workspace, has given up since the last such query (the
 * outputs of that call are undefined), else GPTQ_OK.  It is recorded beside the workspaces' status, which the next call on a workspace resets:
 * a program that runs many calls asks once, after them.  (In a stream that is captured: CUDA.)
 * Errors of its own: CUDA.
 */
gptq_status gptq_serving_status(gptq_stream_t stream);

/*
 * gptq_debug_fp8_matmul_lost_copy, gptq_debug_kv8_attention_lost_copy: test hooks of the bounded
 * device waits, as gptq_debug_hessian_lost_stage.
 *
 * They run gptq_fp8_matmul (without row factors) and gptq_kv8_attention with copy number lost_copy
 * of every CTA left out (of W and A: one for 128 elements of K; of keys: one for 128 tokens, or, up
 * to 32 rows of a cache head, of keys and values in turn, for 64 tokens of a group of warps), and
 * every wait of the kernel limited to wait_ns (1e3 .. 1e10) nanoseconds.  The waits for that copy
 * give up; the kernel records GPTQ_ERR_TIMEOUT in ws and ends with none of its copies and
 * tensor-core operations in flight.  out is then undefined.  Where no CTA has such a copy the call
 * is the regular one.
 * SYNCHRONIZE `stream` and return the device status.  Errors: as the regular calls.
 */
gptq_status gptq_debug_fp8_matmul_lost_copy(const uint8_t *a, int64_t lda, const uint8_t *a_exps,
                                            int64_t ldae, const uint8_t *w, int64_t ldw,
                                            const uint8_t *w_exps, int64_t ldwe, int64_t m,
                                            int64_t n, int64_t k, void *out, int odtype,
                                            int64_t ldo, int64_t lost_copy, uint64_t wait_ns,
                                            void *ws, size_t ws_bytes, gptq_stream_t stream);
gptq_status gptq_debug_kv8_attention_lost_copy(
    const void *q, const int64_t *q_strides, int dtype, int64_t n_seq, int64_t n_new, int n_heads,
    int n_kv, int dim, const uint8_t *k, const uint8_t *v, const uint8_t *k_exps,
    const uint8_t *v_exps, int64_t n_blocks, const int32_t *table, int64_t ld_table,
    int64_t max_blocks, const int32_t *lengths, int causal, float scale, void *out,
    const int64_t *o_strides, int64_t lost_copy, uint64_t wait_ns, void *ws, size_t ws_bytes,
    gptq_stream_t stream);

/* ======================================================================================
 * Feed-forward blocks on quantized layers: what lies between their products, and experts
 * ====================================================================================== */

/* Activation functions, taken in fp32: x, max(x, 0) (NaN stays), x / (1 + exp(-x)),
 * x (1 + erf(x / sqrt 2)) / 2.  (SILU of less than about -87, below 2^-119 in magnitude, is 0.) */
typedef enum gptq_act {
  GPTQ_ACT_NONE = 0, GPTQ_ACT_RELU = 1, GPTQ_ACT_SILU = 2, GPTQ_ACT_GELU = 3
} gptq_act;

/*
 * gptq_fp8_weights (a HOST struct): the weights W [n, k] of a product in 128 x 128 blocks as in
 * gptq_fp8_matmul, or one such matrix for each of several experts.
 *   codes      [n, ld];  exps: [ceil(n / 128), ld_exps];
 *   next_codes, next_exps   elements from one expert's matrix to the next: multiples of 16 and 4 that
 *              are at least n * ld and ceil(n / 128) * ld_exps (read where there are experts alone).
 *   scale, bias   [n] fp32, or [n_experts, n], or NULL (1, 0).
 */
typedef struct gptq_fp8_weights {
  const uint8_t *codes;
  int64_t ld, next_codes;
  const uint8_t *exps;
  int64_t ld_exps, next_exps;
  const float *scale, *bias;
} gptq_fp8_weights;

/*
 * gptq_fp8_linear_workspace_bytes: workspace size of the four products below; rows: m, or
 * n_tokens * top_k.  0 for bad arguments.
 */
size_t gptq_fp8_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k);

/*
 * gptq_fp8_linear: out [m, n] = act(diag(a_scale) A W^T diag(scale) + bias) + residual, summed in
 * fp32 and rounded once to odtype.
 *
 *   a, a_exps, a_scale, out, ws   as in gptq_fp8_matmul.
 *   act        a gptq_act.
 *   residual   [m, ldr] of odtype, or NULL; it may be out itself (with ldr = ldo).
 * Repeated calls give identical results.  Asynchronous; a bounded device wait that gave up is
 * recorded in ws (gptq_workspace_status).  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.
 */
gptq_status gptq_fp8_linear(const uint8_t *a, int64_t lda, const uint8_t *a_exps, int64_t ldae,
                            const float *a_scale, const gptq_fp8_weights *w, int act,
                            const void *residual, int64_t ldr, int64_t m, int64_t n, int64_t k,
                            void *out, int odtype, int64_t ldo, void *ws, size_t ws_bytes,
                            gptq_stream_t stream);

/*
 * gptq_fp8_gated: codes and exponents, by 1 x 128 blocks, of act(G) * U [m, n], where
 * G = diag(a_scale) A Gate^T diag(scale) + bias and U the same of `up`; all in fp32 until it is
 * rounded to the codes.  What is not finite becomes the NaN code.
 * Otherwise as gptq_fp8_linear.
 */
gptq_status gptq_fp8_gated(const uint8_t *a, int64_t lda, const uint8_t *a_exps, int64_t ldae,
                           const float *a_scale, const gptq_fp8_weights *gate,
                           const gptq_fp8_weights *up, int act, int64_t m, int64_t n, int64_t k,
                           uint8_t *codes, int64_t ldc, uint8_t *exps, int64_t lde, void *ws,
                           size_t ws_bytes, gptq_stream_t stream);

/*
 * gptq_moe_route: which top_k experts each token goes to, with which weights, and the tokens of
 * each expert.
 *
 *   s_e = softmax over the token's logits, or 1 / (1 + exp(-logit)).
 *   c_e = s_e + bias_e; without a bias, whose order is that of the logits, these are compared.
 *   groups > 1: the experts fall into `groups` runs of n_experts / groups; a run's value is the sum
 *         of its group_top (1 or 2) largest c, and only the top_groups best runs are looked at.
 *   ids   the top_k experts of largest c, largest first; equals: the lowest index first.  The
 *         choice is that of 64-bit arithmetic: c nearer to one another than fp32 tells are taken
 *         again in fp64.
 *   weights: s of the chosen experts, with renormalize over their sum, times scale.
 * An expert whose logit or bias is not finite is never chosen; where too few are left, the last ids
 * of the token are -1 and their weights 0.  A logit that is not finite adds nothing to the softmax's
 * sum; a bias, finite or not, has no part in the scores: an expert that only its bias leaves out
 * keeps its part of the sum (and so of weights that are not renormalized).
 *
 *   logits     [n_tokens, ld] of dtype (F16, BF16, F32), ld >= n_experts.
 *   bias       [n_experts] fp32 or NULL.   scores: 0 softmax, 1 sigmoid.
 *   ids [n_tokens, top_k] int32, weights [n_tokens, top_k] fp32 out.
 *   offsets [n_experts + 1] int32, order [n_tokens * top_k] int32 out: order lists the assignments
 *              (token * top_k + place among its ids) by expert, in increasing order for each;
 *              expert e has order[offsets[e]] to order[offsets[e + 1] - 1].  -1 after the last.
 *   1 <= top_k <= 32; n_experts <= 1024, groups <= 32, n_tokens * top_k <= 2^22 (else UNSUPPORTED);
 *   groups divides n_experts, 1 <= top_groups <= groups, group_top <= n_experts / groups and
 *   top_k <= top_groups * n_experts / groups; scale finite.
 *   ws         workspace of ws_bytes >= gptq_moe_route_workspace_bytes(n_tokens, n_experts, top_k).
 * Asynchronous.  Errors: INVALID_ARG, WORKSPACE, UNSUPPORTED, CUDA.
 */
size_t gptq_moe_route_workspace_bytes(int64_t n_tokens, int n_experts, int top_k);
gptq_status gptq_moe_route(const void *logits, int dtype, int64_t ld, int64_t n_tokens,
                           int n_experts, int top_k, const float *bias, int scores, int groups,
                           int top_groups, int group_top, int renormalize, float scale,
                           int32_t *ids, float *weights, int32_t *offsets, int32_t *order,
                           void *ws, size_t ws_bytes, gptq_stream_t stream);

/*
 * gptq_fp8_experts_gated: gptq_fp8_gated of the rows of each expert.  Position p of the order takes
 * A's row order[p] / top_k and the weights of the expert e with offsets[e] <= p < offsets[e + 1],
 * and is row p of the codes.
 *   a          [n_tokens, lda];  a_exps, a_scale likewise.
 *   offsets, order   as written by gptq_moe_route for n_experts and n_tokens * top_k.  Offsets are
 *              limited to [0, n_tokens * top_k] and read as increasing; a position whose order
 *              names no row of A is computed as of zeros.
 *   codes, exps   [n_tokens * top_k, ...]; rows from offsets[n_experts] on stay as they are.
 *   n_experts  1 .. 1024 (else UNSUPPORTED).
 * Otherwise as gptq_fp8_gated.
 */
gptq_status gptq_fp8_experts_gated(const uint8_t *a, int64_t lda, const uint8_t *a_exps,
                                   int64_t ldae, const float *a_scale,
                                   const gptq_fp8_weights *gate, const gptq_fp8_weights *up,
                                   int act, int n_experts, const int32_t *offsets,
                                   const int32_t *order, int top_k, int64_t n_tokens, int64_t n,
                                   int64_t k, uint8_t *codes, int64_t ldc, uint8_t *exps,
                                   int64_t lde, void *ws, size_t ws_bytes, gptq_stream_t stream);

/*
 * gptq_fp8_experts: out[order[p]] = act(A_p W_e^T diag(scale_e) + bias_e) for each position p, e its
 * expert: from rows in the experts' order to rows in the tokens'.
 *   a          [rows, lda], as written by gptq_fp8_experts_gated.
 *   out        [rows, ldo] of odtype; rows that no order names stay as they are.  No two positions
 *              may name one row.
 * Otherwise as gptq_fp8_linear.
 */
gptq_status gptq_fp8_experts(const uint8_t *a, int64_t lda, const uint8_t *a_exps, int64_t ldae,
                             const gptq_fp8_weights *w, int act, int n_experts,
                             const int32_t *offsets, const int32_t *order, int64_t rows, int64_t n,
                             int64_t k, void *out, int odtype, int64_t ldo, void *ws,
                             size_t ws_bytes, gptq_stream_t stream);

/*
 * gptq_debug_fp8_gated_lost_copy: test hook of the bounded device waits of the products above, as
 * gptq_debug_fp8_matmul_lost_copy: gptq_fp8_experts_gated, or with n_experts = 0 gptq_fp8_gated
 * (offsets and order are then not read, and top_k is 1), with copy number lost_copy of every CTA (128
 * elements of K of both weights and, of gptq_fp8_gated, of A) left out and every wait limited to
 * wait_ns.  SYNCHRONIZES `stream` and returns the device status.  Errors: as the regular calls.
 */
gptq_status gptq_debug_fp8_gated_lost_copy(
    const uint8_t *a, int64_t lda, const uint8_t *a_exps, int64_t ldae, const gptq_fp8_weights *gate,
    const gptq_fp8_weights *up, int act, int n_experts, const int32_t *offsets,
    const int32_t *order, int top_k, int64_t n_tokens, int64_t n, int64_t k, uint8_t *codes,
    int64_t ldc, uint8_t *exps, int64_t lde, int64_t lost_copy, uint64_t wait_ns, void *ws,
    size_t ws_bytes, gptq_stream_t stream);

/*
 * gptq_moe_combine: out[t] = residual[t] + sum_j weights[t, j] y[t * top_k + j], summed in fp32 in
 * that order and rounded once.  A row whose weight is 0 is left out, whatever it holds.
 *   y [n_tokens * top_k, ldy], residual [n_tokens, ldr] or NULL, out [n_tokens, ldo] of dtype (F16,
 *   BF16 or F32); out may be the residual.   weights [n_tokens, top_k] fp32.   1 <= top_k <= 32.
 * Asynchronous.  Errors: INVALID_ARG, UNSUPPORTED, CUDA.
 */
gptq_status gptq_moe_combine(const void *y, int dtype, int64_t ldy, int64_t n_tokens, int top_k,
                             int64_t d, const float *weights, const void *residual, int64_t ldr,
                             void *out, int64_t ldo, gptq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_GB300_H */
