/*
 * ns.h -- C ABI of libns.so: batched Newton-Schulz orthogonalization on
 * MI355X (gfx950).
 *
 * The operation. Each matrix G (rows x cols, row-major) of a batch is replaced
 * in place by its Newton-Schulz orthogonalization:
 *
 *     X = G / (||G||_F + 1e-7)
 *     if rows > cols: X = X^T                    (X is m x n, m <= n)
 *     repeat `steps` times:  A = X X^T;  B = b A + c A^2;  X = a X + B X
 *     if transposed: X = X^T;  G <- X rounded to the buffer's dtype
 *
 * The pages this library is built from name this operation as the compute
 * that Muon-family optimizers run on every assembled 2-D update matrix
 * (microsoft/dion PR #74, "Fix megabatch_orthogonalize_async hang on empty
 * FSDP2 shards", Fix section, which also states that zero rows stay zero) and
 * rank its cost as max(M,N)*min(M,N)^2 (NVIDIA/Megatron-LM PR #6379, "Balance
 * LayerWise optimizer shards by Newton-Schulz cost, not parameter size",
 * Changes item 1). They give neither the iteration's coefficients nor its
 * normalization; the specification this library implements fixes them: the
 * Frobenius normalization with eps = 1e-7 added to the norm, the orientation
 * rows <= cols, 5 steps and (a, b, c) = (3.4445, -4.7750, 2.0315), which
 * NS_QUINTIC_* below hold.
 *
 * Precision (what the result is computed with, not a promise of bits):
 *  - bf16 matrices with min(rows, cols) > 32: products on bf16 MFMA with fp32
 *    accumulation. X is carried between steps as two bf16 arrays,
 *    X_hi = bf16(X) and X_lo = bf16(X - X_hi), about 17 significant bits; A
 *    and B are stored as bf16 operands (the same bf16 A in b A and in A^2),
 *    with the rounding residues of their diagonals kept in fp32 and added
 *    back (first-order terms in B, the diagonal of B in the update). The
 *    result is rounded to bf16 (round-to-nearest-even). Relative Frobenius
 *    error against an fp64 evaluation of the same iteration: 2.6e-3 on the
 *    dense low-rank 8192 x 6144 batch, 6e-3 to 1e-2 on Gaussian inputs, up
 *    to 1.4e-2 on small nearly square ones; within 2e-2 at 5 steps.
 *  - matrices of either dtype with min(rows, cols) <= 32 (the small-matrix
 *    path, see NS_SMALL_M): the iteration evaluated in fp64 through the m x m
 *    Gram matrix, which reaches the same result up to rounding: with
 *    X_k = Q_k X_0, A_0 = X_0 X_0^T over the n columns, then per step
 *    B'_k = a I + b A_k + c A_k^2, Q_(k+1) = B'_k Q_k and
 *    A_(k+1) = B'_k A_k B'_k on m x m matrices, and finally Q X_0, rounded to
 *    the buffer's dtype.
 *  - fp32 matrices with min(rows, cols) > 32: fp32 arithmetic throughout
 *    (fp32 MFMA), within 1e-4 of the fp64 evaluation for inputs whose
 *    singular values are not exactly zero. On an exactly rank-deficient
 *    input the rounding noise in its null space grows by about a per step,
 *    as in any fp32 evaluation (e.g. 6e-5 after 5 steps, 2e-3 after 8, on a
 *    rank-4 856 x 535 matrix, within 2x of a plain fp32 evaluation).
 *  - Errors grow with the step count: the bounds above are for the 5 steps
 *    of the specification (bf16 Gaussian inputs reached 1.3e-2 to 1.9e-2
 *    after 8 steps in a seeded sweep).
 *  - The tiled path's norm sums squares in fp32 with per-piece power-of-two
 *    scaling, the small path's in fp64, so every finite input normalizes
 *    (entries up to FLT_MAX); an Inf or NaN entry propagates (see
 *    ns_orthogonalize_batched).
 * Zero rows and columns of G come back as exact +0.0, and a matrix gives the
 * same bits alone, in any batch, at any position and with trailing zero rows
 * appended.
 *
 * Threading. Entry points may be called from several host threads; calls
 * that share a (device, stream) pair are serialized on a lock. All GPU work
 * is enqueued on the caller's stream and no entry point waits for the device,
 * except ns_profile_read and ns_release_workspace as documented, and the
 * NS_CHECK debug mode below.
 *
 * Environment (read at every call):
 *   NS_SMALL_M=t  an integer 0..32: matrices with min(rows, cols) <= t take
 *                 the small-matrix path (default 32); others the tiled path.
 *                 Other values are ignored.
 *   NS_CHECK=1    debug mode: the call waits for the stream after every
 *                 kernel launch and returns NS_EHIP naming the first kernel
 *                 that failed.
 */
#ifndef NS_H
#define NS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NS_BF16 = 0, /* bfloat16 storage */
    NS_FP32 = 1  /* float32 storage  */
} ns_dtype;

typedef enum {
    NS_OK = 0,      /* success (work enqueued)                                */
    NS_EINVAL = 1,  /* invalid argument; nothing was enqueued                 */
    NS_EDTYPE = 2,  /* unknown dtype; nothing was enqueued                    */
    NS_ENOMEM = 3,  /* device or host allocation failed; nothing enqueued     */
    NS_EHIP = 4     /* a HIP call or kernel launch failed; see ns_last_error  */
} ns_status;

#define NS_QUINTIC_A 3.4445f
#define NS_QUINTIC_B (-4.7750f)
#define NS_QUINTIC_C 2.0315f

/*
 * Orthogonalize `count` matrices in place.
 *
 *   ptrs    host array of `count` device pointers. ptrs[i] points at matrix i:
 *           shapes[2i] x shapes[2i+1] elements of `dtype`, row-major and
 *           contiguous (leading dimension = cols), aligned to the element
 *           size. Read as G, overwritten with the result. Matrices must not
 *           overlap. A pointer may be NULL only for an empty matrix.
 *   shapes  host array of 2*count int64: (rows, cols) per matrix, each >= 0.
 *           rows == 0 or cols == 0 is an empty matrix (an empty shard): it is
 *           accepted and never touched.
 *   count   number of matrices, >= 0; 0 enqueues nothing.
 *   steps   iterations, >= 0. steps == 0 writes G / (||G||_F + 1e-7).
 *   coeffs  host array of 3 floats (a, b, c) applied at every step; may be
 *           NULL only when steps == 0.
 *   dtype   an ns_dtype; all matrices of a call share it.
 *   stream  a hipStream_t (NULL = the legacy default stream) on the current
 *           device. All work is enqueued on it; the results are complete in
 *           stream order. Host arrays are only read before the call returns.
 *
 * Workspace: the library keeps a device workspace per (device, stream) pair,
 * grown on demand with stream-ordered allocation (hipMallocAsync /
 * hipFreeAsync), plus a cache of up to 64 batch plans keyed by the argument
 * values (shapes, pointers, dtype). Two calls on the same stream are ordered
 * by the stream; calls on different streams use separate workspaces.
 *
 * Never blocks: the call enqueues its work and returns without waiting for
 * the device, however much work is already queued on the stream (the hang
 * and hidden sync point microsoft/dion PR #74, "Fix
 * megabatch_orthogonalize_async hang on empty FSDP2 shards", Concrete repro
 * and review thread, are about). A batch not in the plan cache uploads its
 * descriptors and tile lists from pinned host staging buffers; one still
 * feeding an earlier upload is never waited for: a new buffer is allocated
 * instead, up to 256 MiB of them per (device, stream), past which the call
 * returns NS_ENOMEM (with nothing enqueued) rather than wait.
 *
 * Errors (all reported before anything is enqueued, except NS_EHIP):
 *   NS_EINVAL  negative count, steps or dimension; NULL ptrs/shapes with
 *              count > 0; NULL pointer for a non-empty matrix; a pointer not
 *              aligned to the element size; NULL coeffs with steps > 0; a
 *              dimension above 2^24; a tiled-path matrix (min(rows, cols)
 *              above the small-path threshold) whose padded operand is too large for 32-bit buffer
 *              offsets: with m, n rounded up to multiples of 256 (mp, np),
 *              np x mp x element size must stay below 2 GiB and
 *              np x 256 x element size below 2 GiB (e.g. 32768 x 32768 bf16
 *              or 8192 x 131072 bf16 is rejected; 10240 x 10240 and
 *              8192 x 65536 bf16 are accepted).
 *   NS_EDTYPE  unknown dtype.
 *   NS_ENOMEM  the workspace or the metadata staging cannot be allocated.
 *   NS_EHIP    a HIP call or kernel launch failed.
 * On any error the message is available from ns_last_error(). NaN and Inf
 * propagate unchecked: a NaN entry makes the whole result NaN.
 */
ns_status ns_orthogonalize_batched(void* const* ptrs, const int64_t* shapes,
                                   int32_t count, int32_t steps,
                                   const float* coeffs, int32_t dtype,
                                   void* stream);

/* Longest coefficient schedule ns_orthogonalize_batched_sched accepts. */
#define NS_MAX_SCHEDULE_STEPS 64

/*
 * As ns_orthogonalize_batched, but step s (0-based) uses its own polynomial:
 *
 *   coeffs  host array of 3*steps floats; (coeffs[3s], coeffs[3s+1],
 *           coeffs[3s+2]) are (a, b, c) of step s. May be NULL only when
 *           steps == 0.
 *   steps   0 .. NS_MAX_SCHEDULE_STEPS.
 *
 * With every triple equal to (a, b, c) the result is bit for bit that of
 * ns_orthogonalize_batched with (a, b, c). This serves iterations whose
 * polynomial changes from step to step, e.g. a few quintic steps followed by
 * cubic (1.5, -0.5, 0) steps that converge to the polar factor UV^T.
 * Errors as ns_orthogonalize_batched, plus NS_EINVAL for steps above
 * NS_MAX_SCHEDULE_STEPS.
 */
ns_status ns_orthogonalize_batched_sched(void* const* ptrs, const int64_t* shapes,
                                         int32_t count, int32_t steps,
                                         const float* coeffs, int32_t dtype,
                                         void* stream);

/*
 * As ns_orthogonalize_batched, for matrices that arrive as row blocks: the
 * row shards an all-to-all hands to the rank that orthogonalizes a matrix
 * (microsoft/dion PR #74, "Fix megabatch_orthogonalize_async hang on empty
 * FSDP2 shards", Summary and Fix: shards of a padded split, some of them
 * empty; InternLM/xtuner PR #2069, the ragged exchange that sends each shard
 * at its own length). Matrix i is the vertical concatenation of its
 * nchunks[i] blocks; it is orthogonalized as that whole matrix and the result
 * is written back into the same blocks, so no assembly or split copy is made.
 * Result bits equal those of ns_orthogonalize_batched on the concatenated
 * matrix.
 *
 *   chunk_ptrs  host array of sum(nchunks) device pointers, matrix 0's blocks
 *               first, each block top to bottom. Block k holds chunk_rows[k]
 *               rows of cols[i] elements, row-major and contiguous, aligned
 *               to the element size; NULL only for an empty block.
 *   chunk_rows  host array of sum(nchunks) int64 row counts, each >= 0. A
 *               block of 0 rows (an empty shard) is never touched.
 *   nchunks     host array of `count` int32 block counts, each >= 0.
 *   cols        host array of `count` int64 column counts, each >= 0.
 *   count, steps, coeffs, dtype, stream: as ns_orthogonalize_batched.
 *
 * Blocks must not overlap. Errors as ns_orthogonalize_batched (NS_EINVAL
 * also for a negative block count or block row count, and for a matrix whose
 * rows add up above 2^24).
 */
ns_status ns_orthogonalize_chunked(void* const* chunk_ptrs, const int64_t* chunk_rows,
                                   const int32_t* nchunks, const int64_t* cols,
                                   int32_t count, int32_t steps,
                                   const float* coeffs, int32_t dtype,
                                   void* stream);

/* Device scratch of ns_orthogonalize_batched_noalloc, per device. */
#define NS_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)

/*
 * As ns_orthogonalize_batched (same arguments, results bit for bit the same),
 * for callers that cannot allocate: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation. This call makes no device
 * or pinned-host allocation (no hipMalloc, hipMallocAsync, hipHostMalloc or
 * hipFree of any kind) and never waits for the device.
 *
 * Workspace: a static device array of NS_NOALLOC_SCRATCH_BYTES that each
 * device this library runs on holds until the process ends (reserved when
 * the library's code is loaded on the device). The batch's workspace and
 * metadata must fit it: ns_workspace_bytes(shapes, count, dtype) + 256 <=
 * NS_NOALLOC_SCRATCH_BYTES (e.g. the 32 attention-gate matrices of 24 x 2304,
 * or one 2048 x 6144 bf16 matrix); a larger batch is rejected with NS_EINVAL
 * before anything is enqueued. The metadata goes up through kernel
 * arguments (one small copy kernel per 2 KB).
 *
 * Every call on a device shares that device's array, which keeps the last
 * call's contents: calls that overlap on one device race (two streams, or two
 * host threads); calls on one stream are ordered by it. Nothing in the array
 * needs to start at any value.
 *
 * Errors as ns_orthogonalize_batched, plus NS_EINVAL for a batch that does
 * not fit the scratch array.
 */
ns_status ns_orthogonalize_batched_noalloc(void* const* ptrs, const int64_t* shapes,
                                           int32_t count, int32_t steps,
                                           const float* coeffs, int32_t dtype,
                                           void* stream);

/*
 * Placement of whole matrices onto `world` data-parallel ranks (host-only; no
 * device is touched): which rank orthogonalizes each matrix and where it sits
 * in that rank's shard of its bucket buffer. NVIDIA/Megatron-LM PR #6379,
 * "Balance LayerWise optimizer shards by Newton-Schulz cost, not parameter
 * size", Problem, Changes 1-3 and Notes.
 *
 *   numel        count element counts of the parameters as stored (a GTP
 *                shard's local count), in backprop order.
 *   cost         count Newton-Schulz costs of the full shapes
 *                (ns_compute_cost of the all-gathered matrix; the element count
 *                for a non-matrix parameter).
 *   world        ranks (> 0); bucket_size: element threshold of a bucket
 *                (>= 0); align: shard start alignment in elements (>= 1).
 *   by_cost      1: largest cost first onto the rank with the least cost so far
 *                (loads kept across buckets) among ranks whose shard stays under
 *                1.3 x (bucket numel / world); a matrix that fits nowhere goes to
 *                the rank with the least numel in the bucket. 0: the earlier
 *                rule, largest numel first onto the rank with the least numel.
 *   absorb       1: bucket_size is a soft minimum: once a bucket reaches it, a
 *                further parameter still joins while a least-loaded placement in
 *                backprop order puts it into existing padding. 0: a bucket
 *                closes as soon as it reaches bucket_size.
 *   rank, offset, bucket  count outputs: rank, element offset within that
 *                rank's shard of the bucket, bucket index.
 *   bucket_elems outputs per bucket (room for count entries): elements the
 *                bucket's buffer holds, world x the largest shard.
 *   nbuckets     output: number of buckets.
 *   rank_cost    optional (may be NULL) world outputs: total cost per rank.
 *
 * Returns NS_EINVAL for negative counts/sizes/costs, world < 1, align < 1 or a
 * NULL output; NS_OK otherwise.
 */
ns_status ns_plan_ranks(const int64_t* numel, const int64_t* cost, int32_t count, int32_t world,
                        int64_t bucket_size, int64_t align, int32_t by_cost, int32_t absorb,
                        int32_t* rank, int64_t* offset, int32_t* bucket, int64_t* bucket_elems,
                        int32_t* nbuckets, int64_t* rank_cost);

/*
 * Device workspace bytes a call with these shapes and dtype needs (host-only;
 * touches no device): lets a caller check the footprint before a call. Same
 * validation of shapes/count/dtype as ns_orthogonalize_batched, including the
 * too-large-for-the-tiled-path NS_EINVAL.
 */
ns_status ns_workspace_bytes(const int64_t* shapes, int32_t count,
                             int32_t dtype, size_t* out_bytes);

/*
 * Free the workspace and plan cache held for (current device, stream): the
 * ownership half of the per-stream workspace that ns_orthogonalize_batched
 * grows on demand. Device memory is released with stream-ordered frees on
 * `stream`, so this is safe while earlier calls are in flight; the pinned
 * host staging buffers are freed after a host wait for their pending uploads
 * (the one entry point that waits). Returns NS_OK if nothing was held.
 */
ns_status ns_release_workspace(void* stream);

/* Message of the last non-OK status on the calling thread ("" if none): the
 * error channel of every entry point above. The string stays valid until the
 * thread's next call into the library. */
const char* ns_last_error(void);

/* Library version string. */
const char* ns_version(void);

/*
 * Newton-Schulz cost of a rows x cols matrix, max(M,N) * min(M,N)^2, the
 * model the Megatron-LM page (PR #6379, Changes item 1) ranks work by and the
 * batch scheduler orders matrices by. 0 for an empty matrix, -1 for a
 * negative dimension. Host-only.
 */
int64_t ns_compute_cost(int64_t rows, int64_t cols);

/*
 * Host-only view of the batch plan, for tests and tools.
 *
 * ns_plan_classify: kinds[i] = 0 (empty), 1 (small: min(rows, cols) <= the
 * NS_SMALL_M threshold, the fp64 Gram-form kernel, one workgroup per
 * 512-column slice), 2 (large: tiled MFMA path).
 *
 * ns_plan_tiles: the tile list of one grouped GEMM stage in launch order.
 *   stage 0 = A = X X^T (upper-triangle tiles), 1 = B = bA + cA^2 (same
 *   tiles), 2 = X <- aX + BX (all tiles). Each tile is 4 int32:
 *   (matrix index into the caller's batch, block row, block column, K depth
 *   in elements). Writes min(capacity, total) tiles to `out` (which may be
 *   NULL when capacity is 0) and the total count to *n_tiles.
 *   *tile_size receives the tile edge in elements.
 */
ns_status ns_plan_classify(const int64_t* shapes, int32_t count, int32_t dtype,
                           int32_t* kinds);
ns_status ns_plan_tiles(const int64_t* shapes, int32_t count, int32_t dtype,
                        int32_t stage, int32_t* out, int64_t capacity,
                        int64_t* n_tiles, int32_t* tile_size);

/*
 * Per-kernel timing with HIP events recorded on the call's stream around
 * every launch the library makes while profiling is on.
 *
 * Kinds: 0 norm partial sums, 1 norm finalize, 2 normalize/transpose/pad,
 * 3 X X^T, 4 bA + cA^2, 5 aX + BX (and final write-back), 6 small-matrix
 * fused kernel, 7 steps==0 write-back.
 *
 * ns_profile_enable(1) clears the accumulators and starts recording;
 * ns_profile_enable(0) stops. ns_profile_read waits for every recorded event
 * (a host wait on the events only), then writes, for the first n_kinds kinds,
 * the total milliseconds and the launch count since the last clear.
 */
#define NS_PROFILE_KINDS 8
ns_status ns_profile_enable(int32_t on);
ns_status ns_profile_read(double* total_ms, int64_t* launches, int32_t n_kinds);

/* ---------------------------------------------------------------------------
 * Linear layers in 8 bits: the products that make the matrices above, with
 * the layer's input kept for the backward pass as 8-bit integers (a quarter
 * to a half of its bytes). For a layer Y = X W^T of T tokens, X T x in and
 * W out x in (row-major, as the framework's matrices are):
 *
 *   ns_q8_quantize     X or W -> Xq, Wq: one int8 per value, one scale per row
 *                      (a token of X, an output channel of W)
 *   ns_q8_dequantize   the values back
 *   ns_q8_matmul       Y  = Xq Wq^T                    (forward)
 *   ns_q8_grad_input   dX = dY Wq                      (backward)
 *   ns_q8_grad_weight  G  = beta G + dY^T Xq           (backward), G out x in:
 *                      with beta = 1 a gradient summed over micro-batches,
 *                      with beta = 0.95, say, Muon's momentum: the matrix that
 *                      ns_orthogonalize_batched takes
 *
 * Every call takes a list of layers of any shapes (experts with ragged token
 * counts, some without tokens). Rows may lie at a pitch: element (r, c) of a
 * matrix with pitch ld is at r ld + c, ld >= cols; what lies between a row's
 * end and the next row is neither used nor written. Pitches that are a
 * multiple of 16 bytes with 16-byte aligned matrices take the fast paths.
 *
 * The calls allocate nothing, keep nothing between calls and never wait for
 * the device, so they can be captured into HIP graphs; calls on several
 * streams and host threads are independent as long as they do not share
 * outputs or workspaces. A layer gives the same bits alone, in any list and at
 * any position in it. Host arrays are only read before the call returns.
 * Outputs must not overlap one another (checked) or any input (not checked).
 *
 * Precision:
 *  - ns_q8_matmul: the products and sums are exact integers (int32), which
 *    bounds in_features; the sum is rounded to fp32, multiplied by the two
 *    scales in fp32 and rounded to the output's dtype. A result within the
 *    type's range is returned also where the sum times one scale is past it.
 *  - ns_q8_grad_input, ns_q8_grad_weight: bf16 MFMA with fp32 sums. dY enters
 *    as it is, the 8-bit operand as q s rounded to fp32, in bf16 parts whose
 *    products are added one after the other: two for bf16 outputs (together
 *    off by at most 2^-15 of q s), three for fp32 ones (2^-46). Where the
 *    scales are powers of two (NS_Q8_POW2) one part is exact, and the product
 *    takes about a half or a third of the time. G enters and leaves in fp32
 *    arithmetic, rounded once at the end.
 *  - NaN and Inf propagate: a row with a NaN or Inf quantises to scale NaN and
 *    q = 0, which stands for NaN; an Inf of dY gives the Inf (or, by a q of 0,
 *    the NaN) that it gives by q s.
 */

/* How ns_q8_quantize chooses a row's scale from m = max |x| over the row. */
typedef enum {
    NS_Q8_ABSMAX = 0, /* s = m / 127 rounded to fp32, at least 2^-126            */
    NS_Q8_POW2 = 1    /* s = the smallest power of two >= m / 127, at least
                         2^-126: up to one bit coarser, but q s is a bf16
                         number, which makes the gradients' products faster   */
} ns_q8_scale;

/* A matrix and its 8-bit form. */
typedef struct {
    int64_t rows, cols;   /* each 0 .. 2^24                                    */
    void* values;         /* rows x cols of the call's dtype, aligned to it    */
    int64_t ld_values;    /* pitch in elements                                 */
    int8_t* q;            /* rows x cols                                       */
    int64_t ld_q;         /* pitch in bytes                                    */
    float* scale;         /* rows                                              */
} ns_q8_rows;

/*
 * q = x / s rounded to the nearest integer (ties to even, |q| <= 127), s per
 * row as `mode` says; reads `values`, writes `q` and `scale`.
 *   dtype   of `values` (NS_BF16 or NS_FP32).
 * Errors (nothing enqueued, but for NS_EHIP): NS_EINVAL for a negative count,
 * dimension or one above 2^24, a pitch below cols or above 2^31 - 1, NULL
 * `mats` with count > 0, NULL or misaligned pointers of a non-empty matrix, an
 * unknown mode, outputs that overlap; NS_EDTYPE; NS_EHIP.
 */
ns_status ns_q8_quantize(const ns_q8_rows* mats, int32_t count, int32_t mode, int32_t dtype, void* stream);

/* values = q s, rounded to dtype; reads `q` and `scale`, writes `values`.
 * Errors as ns_q8_quantize. */
ns_status ns_q8_dequantize(const ns_q8_rows* mats, int32_t count, int32_t dtype, void* stream);

/* One layer of a product. Each call reads the members it names and ignores
 * the others. */
typedef struct {
    int64_t tokens, out_features, in_features;
    const int8_t* xq;       /* tokens x in_features                            */
    int64_t ld_xq;
    const float* x_scale;   /* tokens                                          */
    const int8_t* wq;       /* out_features x in_features                      */
    int64_t ld_wq;
    const float* w_scale;   /* out_features                                    */
    const void* dy;         /* tokens x out_features, bf16                     */
    int64_t ld_dy;
    void* out;              /* Y, dX or G                                      */
    int64_t ld_out;
} ns_q8_layer;

/* Longest sum ns_q8_matmul takes: 131071 products of at most 2^14 stay below
 * 2^31. */
#define NS_Q8_MAX_K 131071

/*
 * out[t][o] = x_scale[t] w_scale[o] sum_i xq[t][i] wq[o][i]; out is
 * tokens x out_features of `dtype`. Reads xq, x_scale, wq, w_scale.
 *
 *   workspace, workspace_bytes  device memory of at least the bytes that
 *           ns_q8_workspace_bytes gives for these layers, 16-byte aligned, for
 *           this call alone until it has run (sums split over a long axis
 *           meet there); may be NULL where that is 0. Needs no initial value.
 *
 * Sizes: tokens up to 2^24; out_features and in_features, which are lengths of
 * rows, up to 2^21, in_features here up to NS_Q8_MAX_K. (A gradient without
 * tokens has no dy, and takes out_features up to 2^24.)
 * Errors (nothing enqueued, but for NS_EHIP): NS_EINVAL for a negative count
 * or dimension, a dimension above 2^24, in_features above NS_Q8_MAX_K, a pitch
 * below the row length or above 2^21 (operands and outputs that are not
 * empty), an output of 2^24 or more tiles of 128 x 128, NULL `layers` with
 * count > 0, NULL or misaligned (to the element size) pointers of a non-empty
 * operand, outputs that overlap, a workspace too small or misaligned;
 * NS_EDTYPE; NS_EHIP. A layer with no outputs is never touched.
 */
ns_status ns_q8_matmul(const ns_q8_layer* layers, int32_t count, int32_t dtype, void* workspace,
                       size_t workspace_bytes, void* stream);

/* out[t][i] = sum_o dy[t][o] w_scale[o] wq[o][i]; out is tokens x in_features,
 * bf16. Reads dy, wq, w_scale. Errors as ns_q8_matmul, but for NS_Q8_MAX_K:
 * the sum has up to 2^21 terms, dy's row. */
ns_status ns_q8_grad_input(const ns_q8_layer* layers, int32_t count, void* workspace, size_t workspace_bytes,
                           void* stream);

/* out[o][i] = beta out[o][i] + sum_t dy[t][o] x_scale[t] xq[t][i]; out is
 * out_features x in_features of `dtype` and is not read when beta == 0. A
 * layer without tokens still scales its out. Reads dy, xq, x_scale. Errors as
 * ns_q8_grad_input; the sum has up to 2^24 terms, the tokens. */
ns_status ns_q8_grad_weight(const ns_q8_layer* layers, int32_t count, float beta, int32_t dtype, void* workspace,
                            size_t workspace_bytes, void* stream);

typedef enum { NS_Q8_MATMUL = 0, NS_Q8_GRAD_INPUT = 1, NS_Q8_GRAD_WEIGHT = 2 } ns_q8_op;

/* Workspace that product `op` (an ns_q8_op) of these layers needs (host-only;
 * reads sizes, pitches and the alignment of pointers, never memory). Checks
 * its arguments as the product does. */
ns_status ns_q8_workspace_bytes(int32_t op, const ns_q8_layer* layers, int32_t count, int32_t dtype,
                                size_t* out_bytes);

/* ---------------------------------------------------------------------------
 * Layers in 8-bit floating point with a scale for each block of 128.
 *
 * A matrix of rows x cols is held as q, one 8-bit float a value, and one scale a
 * block: blocks of 1 x 128 values along a row, or squares of 128 x 128. Block b of
 * a row holds its columns 128 b .. 128 b + 127 (the last one what there is). For a
 * layer Y = X W^T of T tokens:
 *
 *   ns_f8_quantize    X, W, dY -> their 8-bit form, that of their transpose, or
 *                     both in one pass over the values
 *   ns_f8_dequantize  the values back
 *   ns_f8_matmul      C = beta C + A B^T:  Y  = X W^T      (forward)
 *                                          dX = dY (W^T)^T  (backward)
 *                                          G  = beta G + dY^T (X^T)^T: the matrix
 *                     that ns_orthogonalize_batched takes
 *
 * A product's operands have the sum's axis along their rows, and their blocks of
 * 128 lie along it: X and dY are quantised as they are for Y and dX, transposed
 * for G (sums over tokens), W as it is for Y and transposed for dX. Squares of W
 * give the same scales and values both ways.
 *
 * Every call takes a list of matrices or products of any shapes (experts with
 * ragged token counts, some without tokens). The calls allocate nothing, keep
 * nothing between calls and never wait for the device, so they can be captured
 * into HIP graphs; calls on several streams and host threads are independent as
 * long as they do not share outputs or workspaces. A list's sizes are host values:
 * ragged counts that are made on the device (ns_route_experts) have to reach the host
 * before they can cut a list, and a graph holds those of its capture. The same call
 * gives the same bits; a matrix quantises to the same ones in any list, while a
 * product's sum over a long axis is cut by how much of the chip its whole list takes:
 * by the list's sizes, scale types and dtype, wherever its tensors lie. Host arrays
 * are only read before the call returns. Outputs must not overlap one another
 * (checked) or any input (not checked). What lies behind a row's end of q up to a
 * multiple of 16 bytes, and behind a block's one-byte scales up to one of 4, may be
 * read, and is not used.
 *
 * Precision:
 *  - quantised values are exact: q is x / s rounded once, to the nearest 8-bit
 *    float, ties to even.
 *  - bf16 products run on the 8-bit MFMA, whose sums are fp32 but which first adds
 *    the products of eight neighbouring k, cut at 2^-13 of the largest one's power of
 *    two: such a group is off by less than 7 2^-13 of its largest product. Typically
 *    1e-5 to 7e-5 of the result's norm, a hundredth of the output's own rounding; where
 *    large products of a group cancel it is what is left that is off by as much of
 *    them. dtype NS_FP32 does not cut.
 *  - fp32 products run on the bf16 MFMA, with q s widened to bf16 (8-bit floats
 *    times a power of two have no more bits), products exact and sums in fp32; a
 *    scale's own 23 bits multiply each block's sum in fp32. Half the rate of the 8-bit
 *    MFMA. Values whose q s lies below 2^-126 may count as 0 there, those from 2^128 on
 *    as Inf, even where the other operand's scale would bring the product back into
 *    range (bf16 products take scales of every size).
 *  - NaN and Inf: a block with a NaN or an Inf quantises to the scale NaN and q = 0,
 *    which stands for NaN. In products a NaN of q or a scale that is NaN or Inf
 *    makes NaN of the outputs that it enters, an Inf of q (e5m2) what it makes in
 *    the formula.
 */
typedef enum {
    NS_F8_E4M3 = 0, /* 4 exponent, 3 mantissa bits, no Inf: up to 448 */
    NS_F8_E5M2 = 1  /* 5 exponent, 2 mantissa bits: up to 57344       */
} ns_f8_format;

/* What a scale is, and how ns_f8_quantize chooses it from m = max |x| of the block
 * and the format's largest number, t = 448 or 57344. */
typedef enum {
    NS_F8_SCALE_FP32 = 0, /* fp32; s = m / t rounded to fp32, at least 2^-126 */
    NS_F8_SCALE_POW2 = 1  /* one byte e, s = 2^(e - 127), 255 for NaN; s = the smallest
                             power of two >= m / t, at least 2^-126. Products take
                             about half the time with it.                       */
} ns_f8_scale;

/* An 8-bit matrix. */
typedef struct {
    int64_t rows, cols;
    const void* q;        /* rows x cols                                        */
    int64_t ld_q;         /* pitch in bytes                                     */
    const void* scale;    /* ceil(cols / 128) x rows, or (squares) ceil(cols / 128)
                             x ceil(rows / 128): the scale of block b of row r at
                             b ld_scale + r, or + r / 128                       */
    int64_t ld_scale;     /* pitch in scales                                    */
    int32_t format;       /* an ns_f8_format                                    */
    int32_t scale_type;   /* an ns_f8_scale                                     */
    int32_t square;       /* 0: blocks of 1 x 128; 1: of 128 x 128              */
    int32_t reserved;     /* not read                                           */
} ns_f8_matrix;

/* A matrix to be quantised. Either q and scale or qt and scale_t may be NULL
 * (not wanted), not both pairs. */
typedef struct {
    int64_t rows, cols;   /* each 0 .. 2^24                                     */
    const void* values;   /* rows x cols of the call's dtype, aligned to it     */
    int64_t ld_values;    /* pitch in elements                                  */
    void* q;              /* rows x cols                                        */
    int64_t ld_q;
    void* scale;          /* ceil(cols / 128) x rows, or x ceil(rows / 128)     */
    int64_t ld_scale;
    void* qt;             /* the transpose: cols x rows                         */
    int64_t ld_qt;
    void* scale_t;        /* ceil(rows / 128) x cols, or x ceil(cols / 128)     */
    int64_t ld_scale_t;
} ns_f8_rows;

/*
 * Quantises `count` matrices into `format`, with scales of `scale_type` for blocks
 * of 1 x 128 of each output's rows, or squares. q and qt are aligned to 16 bytes at
 * pitches of a multiple of 16, scales of one byte to 4 bytes at pitches of a
 * multiple of 4: what the products ask for. What lies between a row's end and the
 * next row is not written.
 *   dtype   of the values (NS_BF16 or NS_FP32).
 * Errors (nothing enqueued, but for NS_EHIP): NS_EINVAL for a negative count,
 * dimension or one above 2^24, a pitch below the row length or above 2^31 - 1,
 * NULL `mats` with count > 0, NULL or misaligned pointers, one of a pair NULL
 * without the other, no output, an unknown format or scale type, `square` neither
 * 0 nor 1, outputs that overlap; NS_EDTYPE; NS_EHIP. A matrix without values is
 * never touched.
 */
ns_status ns_f8_quantize(const ns_f8_rows* mats, int32_t count, int32_t format, int32_t scale_type,
                         int32_t square, int32_t dtype, void* stream);

/* An 8-bit matrix and where its values go. */
typedef struct {
    ns_f8_matrix matrix;
    void* values;         /* rows x cols of the call's dtype, aligned to it     */
    int64_t ld_values;    /* pitch in elements                                  */
} ns_f8_values;

/* values = q s, rounded to fp32 and then to dtype. Errors as ns_f8_quantize. */
ns_status ns_f8_dequantize(const ns_f8_values* mats, int32_t count, int32_t dtype, void* stream);

/* One product: out (a.rows x b.rows) = beta out + A B^T, a.cols == b.cols. A is of
 * either format, B of NS_F8_E4M3. A scale of NaN or Inf makes NaN. */
typedef struct {
    ns_f8_matrix a, b;
    void* out;            /* of the call's dtype, aligned to it                 */
    int64_t ld_out;       /* pitch in elements                                  */
} ns_f8_product;

/*
 * Runs `count` products. out is not read when beta == 0; a product with a.cols == 0
 * (an expert without tokens) still scales its out.
 *
 *   workspace, workspace_bytes  device memory of at least the bytes that
 *           ns_f8_workspace_bytes gives for these products, 16-byte aligned, for
 *           this call alone until it has run; may be NULL where that is 0. Needs no
 *           initial value.
 *
 * Errors (nothing enqueued, but for NS_EHIP): NS_EINVAL for a negative count or
 * dimension, rows above 2^24, cols or a pitch of q or out above 2^21, a pitch of
 * scales above 2^31 - 1, a pitch below the row length, a.cols != b.cols, q not
 * aligned to 16 bytes or at a pitch that is not a multiple of 16, one-byte scales
 * not aligned to 4 bytes or at a pitch that is not a multiple of 4, an output of
 * more than 2^23 - 1 tiles of 128 x 128, NULL or misaligned pointers of a non-empty
 * operand, a format or scale type that is unknown or (B) not offered, outputs that
 * overlap, a workspace too small or misaligned; NS_EDTYPE; NS_EHIP. A product with
 * no outputs is never touched.
 */
ns_status ns_f8_matmul(const ns_f8_product* products, int32_t count, float beta, int32_t dtype, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Workspace that these products need (host-only; reads sizes, never memory).
 * Checks its arguments as ns_f8_matmul does. */
ns_status ns_f8_workspace_bytes(const ns_f8_product* products, int32_t count, int32_t dtype, size_t* out_bytes);

/* ---------------------------------------------------------------------------
 * Experts' router: which experts a token goes to, with what weights, how many
 * tokens each expert gets (the ragged counts of the lists above) and the balance
 * loss that keeps them alike; and the gradient of it all.
 *
 * For the logits l of E experts and T tokens:
 *
 *   p_te    softmax of token t's logits
 *   chosen  its top_k experts by logit, the largest first, ties to the lowest index
 *           (NaN above all). An expert of logit -Inf is never chosen: where fewer are
 *           left, the index is -1 and the weight 0.
 *   w_ti    p of the chosen, or with `normalize` p over the sum of the token's chosen p
 *   n       tokens that count: those of a mask that is not 0 which have an expert. The
 *           others' chosen are all -1, their weights 0, and their p enters nothing.
 *   c_e     tokens that chose e;  P_e = sum of p_te over the tokens that count
 *   loss    E sum_e (c_e / C) (P_e / n), C = sum_e c_e; 0 when n == 0
 *
 * and for gradients dw of the weights and dL of the loss, c held constant:
 *
 *   dl_te = p_te (g_te - sum_j g_tj p_tj),
 *   g_te  = dL (E / n) (c_e / C) + (e chosen as i) h_ti,
 *   h_ti  = dw_ti, or with `normalize` (dw_ti - sum_j dw_tj w_tj) / (sum of chosen p)
 *
 * All arithmetic is in fp32, sums in a fixed order: the same call gives the same bits,
 * and a token's chosen, weights and gradient (given c and n) do not depend on the tokens
 * beside it.
 * p is off by less than (2 R + 60) 2^-24 of itself, R the distance of the row's logits
 * (p below 2^-126 may be 0). NaN and +Inf propagate as the formulas have it. The calls
 * allocate nothing, keep nothing between calls and never wait for the device, so they
 * can be captured into HIP graphs; a layer of experts that cuts its lists by the counts
 * cannot be as a whole, since those sizes are the host's.
 */
#define NS_ROUTE_MAX_EXPERTS 1024
#define NS_ROUTE_MAX_K 16

typedef struct {
    int64_t tokens;        /* 0 .. 2^24                                           */
    int64_t experts;       /* 1 .. NS_ROUTE_MAX_EXPERTS                           */
    const void* logits;    /* tokens x experts of the call's dtype                */
    int64_t ld;            /* pitch in elements                                   */
    const uint8_t* mask;   /* tokens, 0 for one that does not count; or NULL      */
    int32_t top_k;         /* 1 .. NS_ROUTE_MAX_K, at most experts                */
    int32_t normalize;     /* 0 or 1                                              */
    int32_t* chosen;       /* out: tokens x top_k                                 */
    float* weights;        /* out: tokens x top_k                                 */
    int32_t* counts;       /* out: experts                                        */
    float* probs;          /* out: experts, P_e                                   */
    int32_t* routed;       /* out: n                                              */
    float* loss;           /* out                                                 */
} ns_route;

/*
 * Routes the tokens. workspace, workspace_bytes: device memory of at least the bytes
 * that ns_route_workspace_bytes gives, 16-byte aligned, for this call alone until it
 * has run; may be NULL where that is 0. Needs no initial value.
 * Errors (nothing enqueued, but for NS_EHIP): NS_EINVAL for sizes outside the ranges
 * above, a pitch below experts or above 2^31 - 1, NULL or misaligned pointers (logits
 * and chosen, weights may be NULL when tokens == 0), a workspace too small or
 * misaligned; NS_EDTYPE; NS_EHIP.
 */
ns_status ns_route_experts(const ns_route* route, int32_t dtype, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Workspace of ns_route_experts (host-only). */
ns_status ns_route_workspace_bytes(int64_t tokens, int64_t experts, size_t* out_bytes);

typedef struct {
    int64_t tokens, experts;
    const void* logits;       /* as for ns_route_experts                          */
    int64_t ld;
    int32_t top_k, normalize;
    const int32_t* chosen;    /* tokens x top_k; a token whose first is -1 has no
                                 gradient, other indexes outside the experts none of
                                 their own                                        */
    const int32_t* counts;    /* experts: c, of this call's tokens or summed over
                                 ranks, C below 2^31                              */
    const int32_t* routed;    /* n                                                */
    const float* dweights;    /* tokens x top_k; or NULL for none                 */
    const float* dloss;       /* dL; or NULL for none                             */
    void* out;                /* tokens x experts of the call's dtype; may be the
                                 logits, at their pitch                           */
    int64_t ld_out;
} ns_route_grad;

/* The logits' gradient; reads what ns_route_experts left. Errors as there (counts and
 * routed may be NULL when dloss is). */
ns_status ns_route_experts_grad(const ns_route_grad* grad, int32_t dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NS_H */
