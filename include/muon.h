/*
 * muon.h -- C ABI of the one-GPU Muon optimiser step for GB300 (sm_103a).
 *
 * The step is the local part of the distributed Muon update described in
 * "Frontier Pre-training at Microsoft AI" (papercache deepnotes summary),
 * Method details §5 "Scaling Muon to 16K GPUs", resharding steps 1, 3 and 5,
 * and in "Microsoft Reveals MAI-Base-2 Training Recipe" (xiaohu-jiedu),
 * section "How to Make Parameter Updates Faster and More Stable?":
 *   1. update the FP32 momentum in place and cast it to BF16;
 *   2. batch parameters of identical shape;
 *   3. orthogonalise every whole momentum matrix with a symmetry-aware
 *      Newton-Schulz operator;
 *   4. cast the result back to FP32 and apply it to the FP32 weights.
 * The two all-to-all exchanges between the steps move data between GPUs
 * and are not part of this one-GPU library.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers named *_dev are CUDA device pointers owned by the caller; the
 *    library never frees them.  Pointers named *_host are host pointers.
 *  - Matrices are dense, row-major and contiguous.  A group of `count`
 *    matrices of rows x cols is one buffer of count*rows*cols elements.
 *  - "Wide" layout: a matrix with rows > cols is orthogonalised as its
 *    transpose, so the BF16 working copy of every matrix is m x n with
 *    m = min(rows, cols) <= n = max(rows, cols).
 *  - BF16 values travel as uint16_t bit patterns.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Work is enqueued asynchronously; no entry point synchronises
 *    the stream unless it says so.  Kernels are launched with programmatic
 *    stream serialisation: a kernel may be scheduled while the previous
 *    kernel in the stream still runs, but reads and writes global memory
 *    only after that kernel has completed, so stream order is kept.  The
 *    environment variable MUON_PDL=0 turns this off (plain launches).
 *  - Arguments are validated on the host before anything is enqueued: an
 *    invalid argument returns MUON_ERR_INVALID_ARG and launches nothing.
 *  - A handle is bound to the device that was current when it was created
 *    and is not thread-safe.
 *  - Kernels report device-side failures (a bounded wait that expired, a
 *    non-finite norm, a non-finite logit or quantiser input, an index out of
 *    range) through a flag read by muon_last_device_error().
 */
#ifndef MUON_GB300_H_
#define MUON_GB300_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = 1,       /* bad pointer, size, count or value */
  MUON_ERR_NOMEM = 2,             /* workspace allocation failed */
  MUON_ERR_CUDA = 3,              /* a CUDA runtime/driver call failed */
  MUON_ERR_UNSUPPORTED_ARCH = 4,  /* device is not compute capability 10.3 */
  MUON_ERR_TIMEOUT = 5,           /* a bounded device-side wait expired */
  MUON_ERR_NONFINITE = 6,         /* a momentum norm was NaN or Inf */
  MUON_ERR_NO_DEVICE = 7          /* no CUDA device is visible */
} muon_status_t;

typedef struct muon_handle_s* muon_handle_t;

/* One group of same-shape parameters ("Scaling Muon to 16K GPUs",
 * resharding step 2: parameters of identical shape are batched).
 * `update_scale` multiplies the orthogonalised update (1.0 = plain step). */
typedef struct {
  int32_t rows;
  int32_t cols;
  int32_t count;
  float update_scale;
} muon_group_t;

/* Kernel classes, for timing and launch accounting. */
typedef enum {
  MUON_KERNEL_MOMENTUM_CAST = 0,  /* momentum update + BF16 cast + transpose */
  MUON_KERNEL_NORM = 1,           /* per-matrix Frobenius norm finalisation */
  MUON_KERNEL_NS_GRAM = 2,        /* A = alpha X X^T (symmetric storage, see below) */
  MUON_KERNEL_NS_POLY = 3,        /* B' = a I + b A + c A A (same storage as A) */
  MUON_KERNEL_NS_UPDATE = 4,      /* X' = alpha B' X  (= alpha (a X + b A X + c A^2 X)) */
  MUON_KERNEL_APPLY = 5,          /* W = W (1 - lr wd) - lr s O */
  MUON_KERNEL_SCALE = 6,          /* ns_steps == 0: O = X / s */
  MUON_KERNEL_ADAMW = 7,          /* AdamW companion */
  MUON_KERNEL_TRANSPOSE = 8,      /* BF16 transpose (resharded step) */
  MUON_KERNEL_MOE_ROUTE = 9,      /* routing to experts and its backward pass */
  MUON_KERNEL_MOE_PLAN = 10,      /* grouping of slots by expert */
  MUON_KERNEL_MOE_COMBINE = 11,   /* weighted sum of expert rows and its backward pass */
  MUON_KERNEL_FP8_QUANTIZE = 12,  /* FP8 quantisation (rows, blocks, columns) */
  MUON_KERNEL_FP8_PRODUCT = 13,   /* grouped FP8 products, gated ones among them */
  MUON_KERNEL_FP8_WGRAD = 14,     /* grouped FP8 weight gradient */
  MUON_KERNEL_COUNT = 15,         /* classes of muon_kernel_stats_t */
  MUON_KERNEL_LOSS = 15,          /* losses on logits (muon_kernel_class_stats) */
  MUON_KERNEL_CLASSES = 16        /* all of them */
} muon_kernel_t;

typedef struct {
  double total_ms[MUON_KERNEL_COUNT];   /* summed device time per class */
  int64_t launches[MUON_KERNEL_COUNT];  /* launches per class */
  int64_t total_launches;               /* all kernel launches of the handle */
} muon_kernel_stats_t;

/* The same with the first nine classes alone: what muon_kernel_stats of
 * version 0.1.0 wrote, and what the symbol of that name still writes. */
#define MUON_KERNEL_COUNT_V1 9
typedef struct {
  double total_ms[MUON_KERNEL_COUNT_V1];
  int64_t launches[MUON_KERNEL_COUNT_V1];
  int64_t total_launches;               /* of all classes */
} muon_kernel_stats_v1_t;

/* Plan summary of a group list (pure host computation, no GPU needed). */
typedef struct {
  int32_t n_batches;          /* distinct wide shapes (Newton-Schulz batches) */
  int32_t n_chunks;           /* batch chunks that fit the workspace */
  int32_t max_chunk_matrices; /* largest chunk */
  int64_t matrices;           /* total matrices */
  size_t workspace_bytes;     /* device workspace the plan needs */
  double ns_algorithmic_flops;/* sum over matrices of ns_steps*(3 m^2 n + m^3) */
  int64_t launches_per_step;  /* kernel launches one muon_step makes */
} muon_plan_info_t;

/* Default Newton-Schulz configuration: quintic coefficients (a, b, c),
 * 5 iterations and the epsilon added to the Frobenius norm. */
#define MUON_NS_A 3.4445f
#define MUON_NS_B (-4.7750f)
#define MUON_NS_C 2.0315f
#define MUON_NS_STEPS 5
#define MUON_NORM_EPS 1e-7f

/* Human-readable name of a status code (static string, never NULL). */
const char* muon_status_string(muon_status_t status);

/* Text of the last error raised on the calling thread ("" if none). */
const char* muon_last_error_message(void);

/* Library version string. */
const char* muon_version(void);

/* Create a handle on `device` (-1 = the calling thread's current device).
 * `workspace_bytes_max` caps the device workspace the handle may allocate
 * (0 = default of 8 GiB); groups whose whole batch does not fit are
 * processed in chunks (a single matrix always gets room).  The scratch of
 * muon_moe_plan is apart from it, and all of it together within the same
 * cap: a grouping that needs more is refused (NOMEM).  A call that needs a
 * larger workspace frees the one before it, and with it ends the use of
 * captured graphs of the step's calls (not of the grouping's).  No device memory is allocated until first use.
 * Errors: INVALID_ARG (out == NULL), NO_DEVICE, UNSUPPORTED_ARCH (not
 * sm_103), CUDA. */
muon_status_t muon_create(muon_handle_t* out, int32_t device, size_t workspace_bytes_max);

/* Destroy a handle and free its workspace (synchronises the device). */
muon_status_t muon_destroy(muon_handle_t handle);

/* Plan of a group list under a workspace cap, without a GPU.
 * Same group rules as muon_step.  Errors: INVALID_ARG. */
muon_status_t muon_plan_describe(const muon_group_t* groups, int32_t n_groups,
                                 int32_t ns_steps, size_t workspace_bytes_max,
                                 muon_plan_info_t* out);

/* Partition of a group list's whole matrices over `world` data-parallel
 * ranks ("Scaling Muon to 16K GPUs", resharding step 2: after the
 * exchange every GPU holds a subset of complete matrices and orthogonalises
 * them independently, step 3).  Matrices are independent, so each rank
 * steps its own subset with no exchange between ranks.
 * The split is longest-processing-time-first over single matrices: in
 * order of decreasing estimated device time (ns_steps*(3 m^2 n + m^3)
 * algorithmic flops at 1.9 PFLOP/s plus 24 bytes per element at 6.8 TB/s),
 * each matrix goes to the rank with the least estimated time so far.  A
 * rank's matrices of one group are then laid out as one contiguous slice,
 * ranks in order (same loads, since a group's matrices are identical).
 * first_out, count_out: [n_groups * world] host arrays; entry g*world + r
 *   receives the first matrix index and the matrix count of rank r's slice
 *   of group g (count 0: none).  The slices of a group cover it exactly.
 * rank_seconds_out: NULL or [world] host array: each rank's estimated time.
 * Pure host computation, no GPU needed.  Errors: INVALID_ARG (bad groups,
 * ns_steps outside 0..64, world outside 1..65536, NULL outputs). */
muon_status_t muon_partition(const muon_group_t* groups, int32_t n_groups, int32_t ns_steps,
                             int32_t world, int64_t* first_out, int32_t* count_out,
                             double* rank_seconds_out);

/* The whole Muon step on device buffers ("Scaling Muon to 16K GPUs",
 * resharding steps 1, 3, 5; "How to Make Parameter Updates Faster and More
 * Stable?").  For every matrix of every group:
 *   M  <- mu * M + G                          (FP32, in place)
 *   X  <- bf16_rne(M), transposed if rows > cols
 *   s  <- ||M||_F + 1e-7
 *   X  <- X / s; then ns_steps times: A = X X^T; B = b A + c A^2;
 *         X = a X + B X                       (BF16 operands, FP32 accumulate)
 *   W  <- W (1 - lr*wd) - lr * update_scale * fp32(X), transposed back
 * groups:          [n_groups] host array; rows, cols >= 1; count >= 0.
 * momentum_dev:    [n_groups] host array of device pointers, FP32 in/out.
 * grad_dev:        [n_groups] host array of device pointers, FP32 read-only.
 * weights_dev:     [n_groups] host array of device pointers, FP32 in/out.
 * ns_steps:        0..64 (0 applies the normalised BF16 momentum).
 * The three buffers of a group must not overlap each other.
 * Same-wide-shape groups share one Newton-Schulz batch.
 * Errors: INVALID_ARG (NULL pointer with count > 0, bad sizes, non-finite
 * lr/wd/mu, unaligned pointer: 16-byte alignment is required), NOMEM, CUDA. */
muon_status_t muon_step(muon_handle_t handle, const muon_group_t* groups, int32_t n_groups,
                        float* const* momentum_dev, const float* const* grad_dev,
                        float* const* weights_dev, float lr, float wd, float mu,
                        int32_t ns_steps, void* stream);

/* The same step on HOST buffers: copies momentum, gradient and weights to
 * device staging owned by the handle, runs muon_step, copies momentum and
 * weights back, and synchronises `stream` before returning.  Pinned host
 * memory gives asynchronous copies.  Staging is grown on demand. */
muon_status_t muon_step_host(muon_handle_t handle, const muon_group_t* groups, int32_t n_groups,
                             float* const* momentum_host, const float* const* grad_host,
                             float* const* weights_host, float lr, float wd, float mu,
                             int32_t ns_steps, void* stream);

/* ------------------------------------------------------------------
 * Resharded step (ZeRO data parallelism over several GPUs).
 * "Frontier Pre-training at Microsoft AI", Method details §5, resharding
 * pipeline steps 1-5, and "How to Make Parameter Updates Faster and More
 * Stable?" ("batched momentum resharding"): each rank holds a flat shard
 * of every group's FP32 momentum, gradient and weights; it updates and
 * casts its momentum shard (step 1), an all-to-all per group gives every
 * rank the complete matrices muon_partition assigns it (step 2), the owner
 * orthogonalises them (step 3), a second all-to-all returns each shard's
 * update (step 4), and each rank applies it to its weight shard (step 5).
 * The exchanges themselves are collectives of the caller's communication
 * library; these entry points are the local compute between them.  A
 * shard is the element range [shard_begin, shard_end) of a group's flat
 * buffer; matrix k occupies [k E, (k + 1) E) with E = rows * cols.
 * ------------------------------------------------------------------ */

/* Step 1 on a shard: M <- mu M + G in place (FP32, fused multiply-add, the
 * same arithmetic as muon_step), x_shard <- bf16_rne(M) in the shard's
 * flat layout, and sumsq_out[y] <- the sum of M^2 over the shard's piece
 * of matrix shard_begin / E + y, for every matrix the shard touches
 * ((shard_end - 1) / E - shard_begin / E + 1 entries; FP32 per block,
 * FP64 across blocks, rounded to FP32).  momentum_shard, grad_shard:
 * shard_end - shard_begin FP32 (device); x_shard: as many BF16 (device);
 * sumsq_out: device FP32.  Uses the handle's workspace for the block
 * partials.  Errors: INVALID_ARG, NOMEM, CUDA. */
muon_status_t muon_shard_momentum_cast(muon_handle_t handle, int64_t shard_begin,
                                       int64_t shard_end, int64_t matrix_elems,
                                       float* momentum_shard, const float* grad_shard, float mu,
                                       uint16_t* x_shard, float* sumsq_out, void* stream);

/* On the owner of `count` whole wide matrices m x n (x_wide, BF16,
 * contiguous): inv_norm[k] <- 1 / (sqrt(sum of sumsq[k * parts + j] over j)
 * + 1e-7), the partial sums being the pieces' sums of squares gathered
 * from the shards (parts per matrix, zero where a rank held no piece).
 * As in muon_momentum_cast, a norm above 2^60 rescales x_wide by an exact
 * power of two and inv_norm by its inverse; a non-finite norm sets the
 * device error flag (MUON_ERR_NONFINITE).  Errors: INVALID_ARG, CUDA. */
muon_status_t muon_norm_from_sumsq(muon_handle_t handle, int32_t m, int32_t n, int32_t count,
                                   int32_t parts, const float* sumsq, uint16_t* x_wide,
                                   float* inv_norm, void* stream);

/* dst[k] <- src[k]^T for `count` BF16 matrices of rows x cols (both
 * contiguous, device, not overlapping): the owner turns tall matrices wide
 * for the Newton-Schulz products and the updates back.  Errors:
 * INVALID_ARG (sizes as muon_step's groups, NULL, overlap), CUDA. */
muon_status_t muon_transpose_bf16(muon_handle_t handle, int32_t rows, int32_t cols, int32_t count,
                                  const uint16_t* src, uint16_t* dst, void* stream);

/* Step 5 on a shard: W <- W (1 - lr wd) - lr scale fp32(O) over n_elems
 * flat elements (the same arithmetic as muon_step's apply).
 * weights_shard: FP32 in/out; o_shard: BF16 (device).  Errors:
 * INVALID_ARG (n_elems < 0, NULL, non-finite scalars), CUDA. */
muon_status_t muon_shard_apply(muon_handle_t handle, int64_t n_elems, float* weights_shard,
                               const uint16_t* o_shard, float lr, float wd, float scale,
                               void* stream);

/* Page-locked host memory for the buffers of muon_step_host
 * (cudaHostAlloc, portable across devices).  Copies from it run at the
 * host link's rate; on GB300 hosts measured here, memory locked after the
 * fact with cudaHostRegister copied at a fraction of that rate once more
 * than about 8 GiB of it was locked, while memory from this call kept the
 * full rate.  *out receives the pointer (NULL on failure); free it with
 * muon_host_free.  Errors: INVALID_ARG (out == NULL, bytes == 0), NOMEM. */
muon_status_t muon_host_alloc(size_t bytes, void** out);

/* Free memory from muon_host_alloc (NULL is accepted).  Synchronises with
 * copies still reading or writing it.  Errors: CUDA. */
muon_status_t muon_host_free(void* ptr);

/* Shape rules for the update scale (common Muon variants; the pages give
 * no formula).  The factor multiplies each group's own update_scale. */
typedef enum {
  MUON_SCALE_NONE = 0,         /* 1 */
  MUON_SCALE_SQRT_ASPECT = 1,  /* sqrt(max(1, rows / cols)), rows = output dim */
  MUON_SCALE_RMS_MATCH = 2     /* rms_target * sqrt(max(rows, cols)) */
} muon_scale_rule_t;

/* Options of muon_step_ex. */
typedef struct {
  float lr, wd, mu;
  int32_t ns_steps;       /* 0..64 */
  int32_t nesterov;       /* 0: orthogonalise M' ; 1: orthogonalise G + mu*M' */
  const float* coeffs;    /* host, NULL or 3*ns_steps floats: (a, b, c) per iteration */
  int32_t scale_rule;     /* muon_scale_rule_t */
  float rms_target;       /* MUON_SCALE_RMS_MATCH target (<= 0: 0.2) */
} muon_options_t;

/* muon_step with method variants: Nesterov momentum (the matrix
 * orthogonalised, and normed, is U = G + mu*M' with M' the updated
 * momentum), a per-iteration coefficient schedule, and a shape rule for
 * the update scale.  With nesterov = 0, coeffs = NULL and
 * MUON_SCALE_NONE it equals muon_step.  Same buffers and errors as
 * muon_step; INVALID_ARG also for a NULL opts, an unknown rule or
 * non-finite coefficients. */
muon_status_t muon_step_ex(muon_handle_t handle, const muon_group_t* groups, int32_t n_groups,
                           float* const* momentum_dev, const float* const* grad_dev,
                           float* const* weights_dev, const muon_options_t* opts, void* stream);

/* Step 1 alone: momentum update, BF16 cast into wide layout, and the
 * per-matrix inverse scale 1/(||M||_F + 1e-7).
 * momentum_dev:  count*rows*cols FP32, updated in place.
 * grad_dev:      count*rows*cols FP32.
 * x_wide_dev:    count*m*n BF16 output (m = min, n = max of rows, cols).
 * inv_norm_dev:  count FP32 output.
 * A matrix with ||M||_F > 2^60 (about 1.15e18) leaves its x_wide scaled by
 * an exact power of two 2^e (so that its norm is in [1, 2)) and inv_norm by
 * 2^-e: x * inv_norm, the Newton-Schulz input, is unchanged, and the
 * products' FP32 accumulators stay in range.  The same holds inside
 * muon_step and muon_step_ex. */
muon_status_t muon_momentum_cast(muon_handle_t handle, int32_t rows, int32_t cols, int32_t count,
                                 float* momentum_dev, const float* grad_dev, float mu,
                                 uint16_t* x_wide_dev, float* inv_norm_dev, void* stream);

/* Step 3 alone: batched symmetric Newton-Schulz on `count` wide BF16
 * matrices m x n (m <= n), each pre-scaled by inv_norm[i]:
 *   X0 = inv_norm[i] * x[i]; ns_steps times X = a X + (b A + c A^2) X,
 *   A = X X^T.
 * Each iteration is three products, every result rounded to BF16 where
 * it is stored:
 *   Gram    A  = alpha X X^T            (alpha = inv_norm^2 at iteration 0, else 1)
 *   square  B' = a I + b A + c A A      (the linear term folded into B')
 *   update  X' = alpha B' X             (alpha = inv_norm at iteration 0, else 1)
 * Storage of the symmetric A and B': for m > 128 only the 256 x 256 blocks
 * on and above the block diagonal are computed and stored, nothing is
 * mirrored, and a consumer reads a block left of the diagonal as the
 * transpose of the stored block above it; for m <= 128 the matrix is one
 * tile, computed once and stored in full (the part above the diagonal
 * also written mirrored below it).  MUON_NS_PAIR=0 in the environment
 * runs every size on the single-CTA kernels (128-row tiles, stored in
 * full), for comparisons.
 * x_dev, out_dev: count*m*n BF16, 16-byte aligned, must not overlap.
 * inv_norm_dev:   count FP32 (device).
 * coeffs_host:    3 floats (a, b, c) or NULL for the defaults.
 * m and n must be multiples of 8 (row pitch of 16 bytes for the tensor
 * memory accelerator).  Errors: INVALID_ARG, NOMEM, CUDA. */
muon_status_t muon_newton_schulz_bf16(muon_handle_t handle, int32_t m, int32_t n, int32_t count,
                                      const uint16_t* x_dev, uint16_t* out_dev,
                                      const float* inv_norm_dev, int32_t ns_steps,
                                      const float* coeffs_host, void* stream);

/* Step 5 alone: W <- W (1 - lr*wd) - lr*scale*fp32(O), O given in wide
 * layout (transposed back when rows > cols).
 * weights_dev: count*rows*cols FP32 in/out; o_wide_dev: count*m*n BF16. */
muon_status_t muon_apply_update(muon_handle_t handle, int32_t rows, int32_t cols, int32_t count,
                                float* weights_dev, const uint16_t* o_wide_dev,
                                float lr, float wd, float scale, void* stream);

/* Newton-Schulz without any memory allocation (no handle).
 *
 * The pages have no counterpart of this entry point: it exists for callers
 * that cannot allocate device memory at the time they orthogonalise --
 * code running inside CUDA graph construction, custom allocators or
 * runtimes that must not re-enter the CUDA allocator, and deployments
 * whose device memory is fixed at start-up.  It computes what
 * muon_newton_schulz_bf16 computes, with the same arguments and layout,
 * but its scratch (one more m x n iterate plus the m x m matrices A and B
 * per matrix) lives in a file-scope device array of
 * MUON_STATIC_SCRATCH_BYTES (64 MiB) that every GPU loading the library
 * holds until the process exits.  It calls no cudaMalloc, cudaFree or
 * allocating library routine.
 *  - Limit: one matrix must fit the array, i.e.
 *    2*m*n + 4*m*m bytes (each part rounded up to 256) <= 64 MiB - 256;
 *    larger matrices are rejected with MUON_ERR_INVALID_ARG and a message
 *    (muon_last_error_message).  Larger counts are processed in passes.
 *  - First call on a device: resolves the array's device address
 *    (cudaGetSymbolAddress) and sets kernel attributes, with that device
 *    current.  Make that first call before any stream capture.  If that
 *    set-up fails the call returns MUON_ERR_CUDA and the next call on the
 *    device tries the set-up again.
 *  - Sharing: every call uses the same array and leaves its last contents
 *    there; nothing in it needs to start at zero (every scratch element is
 *    written before it is read).  Calls that overlap on the GPU (different
 *    streams, or different host threads) race on the array: serialise them.
 *  - error_flag_dev: optional device int that receives the device error
 *    bits (1 = a bounded wait expired); the caller zeroes it.  With NULL,
 *    the bits go to a word inside the array (cleared at each call) and are
 *    not reported.
 * Errors: INVALID_ARG (shapes as for muon_newton_schulz_bf16, matrix too
 * large for the array, NULL or unaligned buffers, overlap), CUDA. */
#define MUON_STATIC_SCRATCH_BYTES (64u << 20)
muon_status_t muon_newton_schulz_bf16_static(int32_t m, int32_t n, int32_t count,
                                             const uint16_t* x_dev, uint16_t* out_dev,
                                             const float* inv_norm_dev, int32_t ns_steps,
                                             const float* coeffs_host, int32_t* error_flag_dev,
                                             void* stream);

/* Synchronise `stream`, then read and clear the handle's device error
 * flag: MUON_OK, MUON_ERR_TIMEOUT, MUON_ERR_INVALID_ARG (an index read on
 * the device was out of range) or MUON_ERR_NONFINITE. */
muon_status_t muon_last_device_error(muon_handle_t handle, void* stream);

/* AdamW options (decoupled weight decay, bias correction; step >= 1 is the
 * 1-based step count used for the bias corrections). */
typedef struct {
  float lr, beta1, beta2, eps, wd;
  int32_t step;
} muon_adamw_options_t;

/* AdamW companion for the parameters Muon does not handle -- embeddings,
 * norms, scalars ("Microsoft Reveals MAI-Base-2 Training Recipe", section
 * "How to Make Parameter Updates Faster and More Stable?": Muon for 2-D
 * non-embedding matrices, AdamW for the rest).  For every tensor i (FP32,
 * numel[i] elements, device pointers, updated in place except grads):
 *   p <- p (1 - lr wd);  m <- b1 m + (1 - b1) g;  v <- b2 v + (1 - b2) g^2
 *   p <- p - (lr / (1 - b1^step)) m / (sqrt(v) / sqrt(1 - b2^step) + eps)
 * numel: host array; the four pointer arrays are host arrays of device
 * pointers, 4-byte aligned (16-byte alignment enables vector access).
 * Up to 40 tensors per kernel launch; more are launched in batches.
 * Errors: INVALID_ARG (NULL, unaligned, beta outside [0,1), eps <= 0,
 * step < 1, non-finite), CUDA. */
muon_status_t muon_adamw_step(muon_handle_t handle, int32_t n_tensors, const int64_t* numel,
                              float* const* params_dev, const float* const* grads_dev,
                              float* const* exp_avg_dev, float* const* exp_avg_sq_dev,
                              const muon_adamw_options_t* opts, void* stream);

/* ------------------------------------------------------------------
 * The mixture-of-experts layer whose weights the step updates: routing of
 * tokens to experts, grouping of the routed tokens, FP8 products with the
 * experts' weights, and all of it backwards down to FP32 weight gradients
 * in the layout muon_step takes ("Frontier Pre-training at Microsoft AI":
 * 512 routed experts per layer, top-7 routing, training in 8 bits).
 *
 * Of T tokens with k experts each, slot i = t k + j is token t's j-th
 * choice.  muon_moe_plan orders the slots by expert; the r-th of them is
 * row r, and rows [offsets[e], offsets[e+1]) belong to expert e.  Row
 * buffers are as long as there are slots (T k rows); the rows past
 * offsets[experts] (slots without an expert) are neither read nor written.
 * Nothing is copied to the host: the kernels read offsets on the device.
 *
 * FP8 values are e4m3 with one E8M0 scale (the power of two 2^(byte - 127))
 * per 128 values along the summed dimension: not MXFP8, whose scales are per
 * 32 values.  Hidden sizes are multiples of
 * 16 (a last block of fewer than 128 values is allowed); device buffers are
 * 16-byte aligned; inputs and outputs of a call must not overlap.
 *
 * A NaN or an infinity that a router or a quantiser meets sets the device
 * error flag (MUON_ERR_NONFINITE; a logit of -inf is an ordinary mask), an
 * id, row or offset out of range sets it too (MUON_ERR_INVALID_ARG) and is
 * left out: no buffer is read or written outside its bounds.
 * ------------------------------------------------------------------ */

typedef enum { MUON_FP32 = 0, MUON_BF16 = 1 } muon_dtype_t;
typedef enum { MUON_SCORE_SIGMOID = 0, MUON_SCORE_SOFTMAX = 1 } muon_score_t;

/* Options of the routing. */
typedef struct {
  int32_t score;         /* muon_score_t */
  int32_t groups;        /* experts are split into this many equal groups (1..32) */
  int32_t top_groups;    /* only the best of them are chosen from (1..groups) */
  int32_t group_top;     /* a group's value: the sum of its best 1 or 2 choice values */
  int32_t renormalize;   /* divide a token's weights by their sum */
  float scale;           /* then multiply by this */
} muon_route_options_t;

/* Routing of tokens to experts.  With x a token's logits, s_e = sigmoid(x_e)
 * or softmax(x)_e and c_e = s_e + bias_e:
 *   ids[t][j]      the experts of the top_k largest c, largest first, equal
 *                  ones in order of expert, from the top_groups best groups
 *   weights[t][j]  scale s_e, or scale s_e / (sum of the chosen s)
 * A softmax without bias and with group_top 1, or with every group kept,
 * chooses by x itself.  The bias takes part in the choice alone.  An expert whose logit is -inf is
 * closed to the token (so is a NaN or +inf, which is also reported); when
 * fewer than top_k are open, or mask[t] is 0, the slots left over hold id
 * -1 and weight 0.  When every chosen score underflows to zero the
 * renormalised weights are zero.
 * logits: [tokens][experts] of logits_type; bias: [experts] FP32 or NULL;
 * mask: [tokens] bytes or NULL; ids: [tokens][top_k] int32; weights:
 * [tokens][top_k] FP32.  experts 1..1024, top_k 1..min(32, experts).
 * Errors: INVALID_ARG (sizes, groups not dividing experts, fewer than top_k
 * experts in top_groups groups, scale not finite), CUDA. */
muon_status_t muon_moe_route(muon_handle_t handle, int64_t tokens, int32_t experts, int32_t top_k,
                             const void* logits, int32_t logits_type, const float* bias,
                             const uint8_t* mask, const muon_route_options_t* opts, int32_t* ids,
                             float* weights, void* stream);

/* Its backward pass: the gradient of the logits (their type) from that of
 * the weights (grad_weights: [tokens][top_k] FP32), the choice held fixed.
 * Every element of grad_logits is written; slots of -1 contribute nothing.
 * ids as muon_moe_route gave them (distinct experts per token).  Only
 * score, renormalize and scale of opts matter. */
muon_status_t muon_moe_route_backward(muon_handle_t handle, int64_t tokens, int32_t experts,
                                      int32_t top_k, const void* logits, int32_t logits_type,
                                      const int32_t* ids, const float* grad_weights,
                                      const muon_route_options_t* opts, void* grad_logits,
                                      void* stream);

/* Grouping of slots by expert (a stable counting sort).  ids: [n_slots],
 * -1 for none.  offsets: [experts + 1]; slots: [n_slots], the slot of each
 * row, -1 past offsets[experts]; pos: [n_slots], the row of each slot or
 * -1.  More than 2048 slots take scratch of the handle's, allocated at the
 * first such call (512 KiB: enough for 2^20 slots) and again where a call
 * needs more; none of it is freed before the handle, so a captured call stays
 * valid whatever the handle does later.  Calls on several streams that use it
 * are ordered by the caller.  Past 2^20 slots every block adds up the
 * histograms of all blocks, and the time grows faster than their number:
 * 2^20 slots 31 us, 2^22 132 us, 2^24 0.9 ms, 2^26 11 ms (512 experts).
 * Errors: INVALID_ARG, NOMEM, CUDA. */
muon_status_t muon_moe_plan(muon_handle_t handle, int64_t n_slots, int32_t experts,
                            const int32_t* ids, int32_t* offsets, int32_t* slots, int32_t* pos,
                            void* stream);

/* out[t] = sum over j of weights[t][j] y[pos[t][j]] (slots of -1 left out;
 * weights NULL: ones, the backward pass of sending a token to its rows).
 * y: [rows][hidden] BF16; out: [tokens][hidden] BF16, summed in FP32 in the
 * order of j and rounded once. */
muon_status_t muon_moe_combine(muon_handle_t handle, int64_t tokens, int32_t top_k, int64_t rows,
                               int32_t hidden, const uint16_t* y, const int32_t* pos,
                               const float* weights, uint16_t* out, void* stream);

/* Its backward pass: grad_y[pos[t][j]] = weights[t][j] grad_out[t] and
 * grad_weights[t][j] = <grad_out[t], y[pos[t][j]]> (0 for a slot of -1).
 * grad_weights NULL: not wanted (y may then be NULL). */
muon_status_t muon_moe_combine_backward(muon_handle_t handle, int64_t tokens, int32_t top_k,
                                        int64_t rows, int32_t hidden, const uint16_t* grad_out,
                                        const uint16_t* y, const int32_t* pos,
                                        const float* weights, uint16_t* grad_y,
                                        float* grad_weights, void* stream);

/* FP8 quantisation.  Of a block of 128 values with largest magnitude m the
 * scale is the least power of two with m / scale <= 448 (1 for zeros), and
 * q = e4m3(x / scale) to nearest even; NaN stays NaN, infinities saturate.
 *
 * Rows: blocks run along a row of x [tokens][hidden] (BF16).  pos NULL: q
 * [tokens][hidden], scales [tokens][ceil(hidden / 128)].  Otherwise row t is
 * written to the rows pos[t][j] >= 0 of q and scales (`rows` of them).
 * live_rows: NULL, or one int32 on the device (offsets + experts, say; 4-byte
 * aligned, outside q and scales): only that many first rows of x are read and
 * written, whatever the others hold (with pos they are tokens, which
 * muon_moe_plan's offsets do not count). */
muon_status_t muon_fp8_quantize_rows(muon_handle_t handle, int64_t tokens, int32_t hidden,
                                     const uint16_t* x, const int32_t* pos, int32_t top_k,
                                     int64_t rows, const int32_t* live_rows, uint8_t* q,
                                     uint8_t* scales, void* stream);

/* Weights w [experts][n][k] (w_type), one scale per 128 x 128 block: q
 * [experts][n][k] with scales [experts][ceil(n / 128)][ceil(k / 128)], and
 * the transpose qt [experts][k][n] with scales_t transposed alike.  Either
 * pair may be NULL. */
muon_status_t muon_fp8_quantize_blocks(muon_handle_t handle, int32_t experts, int32_t n, int32_t k,
                                       const void* w, int32_t w_type, uint8_t* q, uint8_t* scales,
                                       uint8_t* qt, uint8_t* scales_t, void* stream);

/* Columns of each expert's rows, for the weight gradient, whose sums run
 * over rows: blocks of 128 rows of one expert, written transposed.  An
 * expert's columns of qt [hidden][capacity] start at 128 times the sum of
 * ceil(rows / 128) over the experts before it; they hold its rows, then zeros
 * to the next multiple of 32, and what is left of its last 128 is not written
 * (muon_fp8_grouped_wgrad does not use it), nor are columns past the last
 * expert's.  scales: [capacity / 128][hidden].  capacity is a multiple of
 * 128; rows + 127 experts, rounded down to one, always suffices (0 for no
 * rows: muon_fp8_grouped_wgrad takes that too).  Row r is
 * x[r] of x [x_rows][hidden] (BF16), or x[slots[r] / top_k] with slots [rows]
 * from muon_moe_plan. */
muon_status_t muon_fp8_quantize_cols(muon_handle_t handle, int64_t x_rows, int32_t hidden,
                                     const uint16_t* x, int32_t experts, const int32_t* offsets,
                                     int64_t rows, const int32_t* slots, int32_t top_k, uint8_t* qt,
                                     int64_t capacity, uint8_t* scales, void* stream);

/* Grouped FP8 product: y[r] = x[r] w[e]^T for the rows r of each expert e,
 * FP32 accumulation, rounded once to BF16.  x [rows][k] and x_scales as
 * muon_fp8_quantize_rows gives them, w [experts][n][k] and w_scales as
 * muon_fp8_quantize_blocks does; y [rows][n].  The forward pass takes w, the
 * gradient of its input the transposed weights.  One expert over all rows
 * is a dense product.  k and n multiples of 16. */
muon_status_t muon_fp8_grouped_matmul(muon_handle_t handle, int64_t rows, int32_t experts,
                                      int32_t n, int32_t k, const uint8_t* x,
                                      const uint8_t* x_scales, const uint8_t* w,
                                      const uint8_t* w_scales, const int32_t* offsets, uint16_t* y,
                                      void* stream);

/* The gated feed-forward block of the experts (one expert: a dense block), whose
 * activation is act = f(gate) * up with f one of these (s: the logistic
 * function): x s(x); x s(2 sqrt(2 / pi) (x + 0.044715 x^3)), which is
 * x (1 + tanh(...)) / 2; max(x, 0). */
typedef enum { MUON_GATE_SILU = 0, MUON_GATE_GELU = 1, MUON_GATE_RELU = 2 } muon_gate_t;

/* Forward, both projections and the activation in one kernel: gate[r] =
 * x[r] w_gate[e]^T, up[r] = x[r] w_up[e]^T, act[r] = f(gate[r]) up[r] for the
 * rows r of each expert e.  x and the weights as muon_fp8_grouped_matmul takes
 * them; act [rows][n] BF16, rounded once from the FP32 sums.  gate and up
 * [rows][n] BF16: for the backward pass, or both NULL.  activation: muon_gate_t. */
muon_status_t muon_gated_fp8_matmul(muon_handle_t handle, int64_t rows, int32_t experts, int32_t n,
                                    int32_t k, const uint8_t* x, const uint8_t* x_scales,
                                    const uint8_t* w_gate, const uint8_t* gate_scales,
                                    const uint8_t* w_up, const uint8_t* up_scales,
                                    const int32_t* offsets, int32_t activation, uint16_t* act,
                                    uint16_t* gate, uint16_t* up, void* stream);

/* Backward, the product and the derivatives in one kernel: with g[r] =
 * x[r] w[e]^T (x: the gradient of the down projection's output, quantised; w
 * [experts][n][k]: its weights transposed) and the gate and up that the forward
 * pass wrote,
 *   grad_gate = g up f'(gate), grad_up = g f(gate), act = f(gate) up
 * each [rows][n] BF16, rounded once (f'(0) = 0 of max(x, 0)).  act, for the down
 * projection's weight gradient, may be NULL: it is made again from the rounded gate
 * and up, so that the forward pass's need not be kept. */
muon_status_t muon_gated_fp8_backward(muon_handle_t handle, int64_t rows, int32_t experts,
                                      int32_t n, int32_t k, const uint8_t* x,
                                      const uint8_t* x_scales, const uint8_t* w,
                                      const uint8_t* w_scales, const int32_t* offsets,
                                      int32_t activation, const uint16_t* gate, const uint16_t* up,
                                      uint16_t* grad_gate, uint16_t* grad_up, uint16_t* act,
                                      void* stream);

/* y[r] = x1[r] w1[e]^T + x2[r] w2[e]^T, the sum in FP32, rounded once to BF16: the
 * block's input gradient from grad_gate, grad_up and the transposed projections.
 * Both products have the same n and k; operands as for muon_fp8_grouped_matmul. */
muon_status_t muon_gated_fp8_matmul_sum(muon_handle_t handle, int64_t rows, int32_t experts,
                                        int32_t n, int32_t k, const uint8_t* x1,
                                        const uint8_t* x1_scales, const uint8_t* w1,
                                        const uint8_t* w1_scales, const uint8_t* x2,
                                        const uint8_t* x2_scales, const uint8_t* w2,
                                        const uint8_t* w2_scales, const int32_t* offsets,
                                        uint16_t* y, void* stream);

/* Grouped FP8 weight gradient: dw[e] = dY[e]^T X[e] over the rows of each
 * expert, FP32 (with accumulate: added to dw).  yt [n][capacity] and xt
 * [k][capacity] with their scales as muon_fp8_quantize_cols gives them for
 * these offsets; dw [experts][n][k], the layout of muon_step's gradients.
 * An expert without rows gets zeros (or keeps what it has); with a capacity
 * of 0 that is all of them, and yt, xt and their scales may be NULL. */
muon_status_t muon_fp8_grouped_wgrad(muon_handle_t handle, int32_t experts, int32_t n, int32_t k,
                                     int64_t capacity, const uint8_t* yt, const uint8_t* yt_scales,
                                     const uint8_t* xt, const uint8_t* xt_scales,
                                     const int32_t* offsets, float* dw, int32_t accumulate,
                                     void* stream);

/* ------------------------------------------------------------------
 * Losses on logits, with the gradient of the logits: what a training step
 * starts its backward pass from.
 *
 * logits: [tokens] rows of `vocab` values of logits_type, `ld` >= vocab
 * elements apart, at any element's address (1 <= vocab <= 2^24, tokens <=
 * 2^27); -inf is an ordinary mask.  With q = softmax(z / temperature) and
 * lse = log sum exp(z / temperature), the loss of a token comes with its
 * lse (both FP32).  mask: [tokens] bytes or NULL; a token whose mask is 0 is
 * left out: its logits are not read, its loss, lse and gradient are 0.
 *
 * The gradient, of the logits' type, is that of sum_t grad_loss[t] loss[t]
 * (mean, token weights and loss scaling are in grad_loss, FP32).  Where
 * grad_loss is known beforehand, a call with grad_loss and grad_logits makes
 * loss and gradient together and reads the logits once (where both are NULL,
 * the loss alone); the _backward calls make the gradient later from the lse.
 * (They have q from the lse as FP32 holds it: a gradient's relative error is half a
 * step of the lse, 5e-7 at 12; logits past 2^20 times the temperature, whose lse has
 * steps of 1/8 and more, want the call that makes both.)
 * grad_logits: `grad_ld` elements apart, every element of every row written;
 * it may be the logits themselves (the same address and pitch), and overlaps
 * no other buffer.  (Vectors are stored where its rows start at the same
 * place within 16 bytes as the logits', single elements otherwise.)
 *
 * A loss or lse that is not finite is written as it is and sets the device
 * error flag (MUON_ERR_NONFINITE): NaN where the logits or the teacher's have no
 * softmax (a NaN or +inf among them, logits of -inf alone; the lse alone where the
 * policy loss does not depend on it), an infinity for a target whose q is 0.  An id outside the vocabulary sets it too (MUON_ERR_INVALID_ARG) and is
 * left out.  Buffers are aligned to their elements; inputs and outputs must not
 * overlap but for grad_logits, where rows with a pitch count as one stretch from the
 * first element to the last (a gradient in the gaps between the logits' rows is
 * refused).  No call takes device memory.
 * ------------------------------------------------------------------ */

/* Options of the distillation. */
typedef struct {
  float temperature;     /* of both softmaxes (1e-4 to 1e4) */
  float scale;           /* factor of the loss (temperature^2 keeps gradients' size) */
} muon_distill_options_t;

/* Distillation from a teacher's top logits: with p the softmax of a token's
 * teacher logits over the temperature,
 *   loss[t] = scale sum_j p_j (log p_j - log q[ids[t][j]])
 * teacher: [tokens][targets] of teacher_type; ids: [tokens][targets] int32,
 * the vocabulary entry of each, -1 for none (so is a teacher logit of -inf);
 * equal ids of a token add up, each with its own p_j log p_j.  A token without any target is
 * left out.  One target per token is cross entropy.  targets 1..1024.
 * Errors: INVALID_ARG, CUDA. */
muon_status_t muon_distill_loss(muon_handle_t handle, int64_t tokens, int32_t vocab,
                                const void* logits, int32_t logits_type, int64_t ld,
                                int32_t targets, const void* teacher, int32_t teacher_type,
                                const int32_t* ids, const uint8_t* mask,
                                const muon_distill_options_t* opts, float* loss, float* lse,
                                const float* grad_loss, void* grad_logits, int64_t grad_ld,
                                void* stream);
muon_status_t muon_distill_loss_backward(muon_handle_t handle, int64_t tokens, int32_t vocab,
                                         const void* logits, int32_t logits_type, int64_t ld,
                                         int32_t targets, const void* teacher,
                                         int32_t teacher_type, const int32_t* ids,
                                         const uint8_t* mask, const muon_distill_options_t* opts,
                                         const float* lse, const float* grad_loss,
                                         void* grad_logits, int64_t grad_ld, void* stream);

/* Options of the policy loss. */
typedef struct {
  float temperature;     /* of the softmax (1e-4 to 1e4) */
  float clip_low;        /* the ratio is clipped to 1 - clip_low (0 to 1) ... */
  float clip_high;       /* ... 1 + clip_high (0 or more) */
  float kl_coef;         /* factor of the KL term */
} muon_policy_options_t;

/* Clipped policy loss of a token's action a: with logp = log q_a,
 * r = exp(logp - old_logp) and d = ref_logp - logp,
 *   loss[t] = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *             + kl_coef (exp(d) - d - 1)
 * where A = advantages[t]; a ratio that equals a bound is not clipped.
 * actions: [tokens] int32, -1 for a token without one (left out, as by the
 * mask; its logp is 0); advantages, old_logp, ref_logp: [tokens] FP32.
 * old_logp NULL: the policy that acted is this one (r = 1, and its
 * gradient A); ref_logp NULL: no KL term.  logp: [tokens] FP32, an output of
 * the loss and an input of its backward pass, which clips by it.
 * Errors: INVALID_ARG, CUDA. */
muon_status_t muon_policy_loss(muon_handle_t handle, int64_t tokens, int32_t vocab,
                               const void* logits, int32_t logits_type, int64_t ld,
                               const int32_t* actions, const float* advantages,
                               const float* old_logp, const float* ref_logp, const uint8_t* mask,
                               const muon_policy_options_t* opts, float* loss, float* logp,
                               float* lse, const float* grad_loss, void* grad_logits,
                               int64_t grad_ld, void* stream);
muon_status_t muon_policy_loss_backward(muon_handle_t handle, int64_t tokens, int32_t vocab,
                                        const void* logits, int32_t logits_type, int64_t ld,
                                        const int32_t* actions, const float* advantages,
                                        const float* old_logp, const float* ref_logp,
                                        const uint8_t* mask, const muon_policy_options_t* opts,
                                        const float* logp, const float* lse,
                                        const float* grad_loss, void* grad_logits,
                                        int64_t grad_ld, void* stream);

/* Failure-path self-test of the bounded device waits: launches one small
 * kernel that waits, through the same wait routine the Newton-Schulz
 * kernels use, on a barrier nothing will complete.  The wait gives up after
 * `limit_ms` (1..2000), sets the handle's device error flag and the kernel
 * returns normally, leaving the context usable; muon_last_device_error()
 * then reports MUON_ERR_TIMEOUT.  No fault, trap or hang is involved.
 * Errors: INVALID_ARG (limit out of range), CUDA. */
muon_status_t muon_selftest_bounded_wait(muon_handle_t handle, int32_t limit_ms, void* stream);

/* The same of the losses that stream rows (loss and gradient in one call, two rows
 * and more for every block): in the handle's next such call nothing brings a
 * block's logits (`what` 1), or what else a row needs (2), after its first row.
 * The waits give up after 2 seconds, the rows that were complete stay, no other is
 * written, and muon_last_device_error() reports MUON_ERR_TIMEOUT.  A call of few rows
 * takes the request off and runs as ever.  Errors: INVALID_ARG. */
muon_status_t muon_selftest_loss_wait(muon_handle_t handle, int32_t what);

/* Per-kernel timing: when enabled, every launch is bracketed by CUDA
 * events on the launching stream.  muon_kernel_stats synchronises the
 * device, folds the recorded events into `out` and keeps accumulating;
 * muon_reset_kernel_stats clears the totals.
 * The symbol muon_kernel_stats keeps the layout it had with nine classes, so
 * that programs built against that header run on; sources that include this
 * one call muon_kernel_stats_v2, with every class, under the same name. */
muon_status_t muon_set_kernel_timing(muon_handle_t handle, int32_t enable);
muon_status_t muon_kernel_stats(muon_handle_t handle, muon_kernel_stats_v1_t* out);
muon_status_t muon_kernel_stats_v2(muon_handle_t handle, muon_kernel_stats_t* out);
#define muon_kernel_stats muon_kernel_stats_v2
muon_status_t muon_reset_kernel_stats(muon_handle_t handle);
/* The same of one class, muon_kernel_stats_t's and those added since
 * (0 <= kind < MUON_KERNEL_CLASSES); either output may be NULL. */
muon_status_t muon_kernel_class_stats(muon_handle_t handle, int32_t kind, double* total_ms,
                                      int64_t* launches);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* MUON_GB300_H_ */
