/*
 * muon.h — C ABI of libmuon.so: the Muon optimizer step for 2-D weight
 * matrices on NVIDIA B200 (sm_100a).
 *
 * The method.  Muon is the orthogonalised-momentum optimizer for matrix
 * parameters ("把 GPT-2 的训练租金估算从 4.3 万美元压到 40 美元 ...",
 * magicnetworld, glossary table, row "Muon"); the hybrid recipe orthogonalises
 * the matrix parameters by Newton-Schulz and leaves the rest to AdamW
 * ("开发者千美元训3.8B模型 击败GPT-2", aiproducthub, 影响 paragraph).  The pages
 * print no formula; the step implemented here, per matrix W, G, M of shape
 * rows x cols, is
 *
 *   M1 = beta*M + (1-beta)*G                         (momentum, lerp form)
 *   U  = (1-beta)*G + beta*M1  if nesterov, else M1  (Nesterov blend)
 *   X  = U, or U^T if rows > cols;  X = X / (||X||_F + eps)
 *   k times:  A = X X^T;  B = b*A + c*A A;  X = a*X + B X
 *   O  = X, or X^T if rows > cols
 *   W1 = (1 - lr*weight_decay)*W - lr*sqrt(max(1, rows/cols))*O
 *
 * Memory.  The caller owns every byte of device memory: W, G, M and one
 * workspace buffer sized by muon_workspace_size().  The library never calls
 * cudaMalloc/cudaFree.  A handle owns only host-side tables (the shape
 * grouping and the TMA descriptors of the workspace).
 *
 * Streams.  muon_step and muon_orthogonalize only enqueue work on the given
 * stream and return; they never synchronise the device, so they can be
 * captured into a CUDA graph.  Pointers must stay valid until the enqueued
 * work has finished.  Calls on one handle must not overlap on the device
 * (they share the workspace).
 *
 * Kernels.  A step enqueues the momentum/norm kernel, then the Newton-Schulz
 * iterations, then the parameter write.  In MUON_MODE_FAST the iterations run
 * as three tensor-core launches each (Gram, polynomial, update) over every
 * matrix of the handle, with the parameter write fused into the last update
 * for bf16 sets whose dimensions are multiples of 32 and whose parameters are
 * 16-byte aligned (the fused write and the separate write kernel compute the
 * same W, bit for bit, from X_k rounded to bf16).  When every matrix fits
 * one 256 x 256 tile (max(rows, cols) <= 256, at most six distinct shapes),
 * all k iterations run in one launch instead (MUON_KERNEL_NS_SMALL).
 * Results are the same function of the inputs on either path, within the
 * bf16 rounding described under muon_mode_t.
 *
 * Errors.  Every entry point returns a muon_status_t and never throws.
 * Argument errors are detected on the host before anything is enqueued.
 * Launch failures return MUON_ERR_CUDA.  Faults the kernels detect on the
 * device (a bounded wait that ran out) are recorded in a status word in the
 * workspace and reported by muon_get_status().
 */
#ifndef MUON_H_
#define MUON_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define MUON_API __attribute__((visibility("default")))
#else
#define MUON_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = 1,    /* null pointer, bad size or count, bad hyper-parameter */
  MUON_ERR_UNSUPPORTED = 2,    /* dtype/mode combination or shape this build does not run */
  MUON_ERR_CUDA = 3,           /* a CUDA runtime/driver call failed (launch, descriptor encode) */
  MUON_ERR_WORKSPACE = 4,      /* workspace null, too small or not 1024-byte aligned */
  MUON_ERR_TIMEOUT = 5,        /* a device-side bounded wait ran out (see muon_get_status) */
  MUON_ERR_DEVICE_STATUS = 6,  /* any other fault recorded by a kernel */
  MUON_ERR_NO_DEVICE = 7       /* no sm_100 device current */
} muon_status_t;

/* Storage type of W, G, M (and of the X/O buffers of muon_orthogonalize).  MUON_FP16 is a type of
 * views only (muon_view_t); a handle's own type is bf16 or fp32. */
typedef enum { MUON_BF16 = 0, MUON_FP32 = 1, MUON_FP16 = 2 } muon_dtype_t;

/* Arithmetic of the Newton-Schulz products.
 * FAST:     bf16 operands on the tcgen05 tensor cores, fp32 accumulation in
 *           TMEM, fp32 epilogue math, one bf16 rounding per stored intermediate
 *           (X, A, and B' = a I + b A + c A A, every term of B' taken from the
 *           rounded A).
 * FP32_REF: fp32 operands and intermediates, products accumulated in fp64 on
 *           the CUDA cores (no TF32): a slow, accurate mode for checking.
 * HALF:     the products of FAST with fp16 operands: three more significant bits in the
 *           same tensor-core instructions, an error about eight times smaller (2e-3 instead of
 *           1-2e-2 after five quintic iterations).  A call takes about as long as in FAST
 *           (measured from 6 % less to 9 % more; 23 % more in a step on 64 of 256 x 256).
 *           X and A are stored times 2^12, so iterations whose singular values stay below 4
 *           are in range (the usual ones stay below 1.3); beyond that a matrix comes out not
 *           finite.  X is normalised before it is rounded, so the inputs' size does not
 *           matter: from norms of about 1e-4 eps (2^-100 with eps = 0) up to the largest fp32
 *           entries.  The norm itself is reported as fp32, so as infinity beyond 3.4e38.  A
 *           matrix that is not finite comes out as NaN.  Matrices of at most 128 rows (or
 *           columns) and 4096 columns (rows), or of fewer rows and as many times more
 *           columns, run every iteration on chip.  Takes views, coefficients per iteration
 *           and 8-bit momentum (below). */
typedef enum { MUON_MODE_FAST = 0, MUON_MODE_FP32_REF = 1, MUON_MODE_HALF = 2 } muon_mode_t;

typedef struct { int64_t rows, cols; } muon_shape_t;

typedef struct {
  float lr;            /* learning rate */
  float beta;          /* momentum coefficient, 0 <= beta <= 1 */
  float weight_decay;  /* decoupled weight decay, applied to the pre-update W */
  float eps;           /* added to ||X||_F before dividing, >= 0; an all-zero X with
                          eps = 0 is taken as the zero direction (zero update) */
  float a, b, c;       /* Newton-Schulz polynomial a x + b x^3 + c x^5 */
  int32_t nesterov;    /* nonzero: Nesterov blend */
  int32_t ns_steps;    /* iterations k, 0 <= k <= 64 */
} muon_hparams_t;

typedef struct muon_ctx* muon_handle_t;

/* Largest number of matrices one handle accepts. */
#define MUON_MAX_MATRICES 4096

/*
 * Bytes of device workspace a handle for these shapes needs.  Matrices of one
 * orientation-free shape (min(rows,cols), max(rows,cols)) form one group and
 * share one batched buffer set; each group holds two X buffers, A and B, all
 * padded with zeros to multiples of 256.
 *   shapes: host array of n shapes, rows >= 1, cols >= 1.
 *   bytes:  host out-pointer.
 * Returns MUON_ERR_INVALID_ARG on a null pointer, n < 1 or n > MUON_MAX_MATRICES,
 * or a dimension below 1 or above 2^20.
 */
MUON_API muon_status_t muon_workspace_size(const muon_shape_t* shapes, int n, muon_dtype_t dtype,
                                  muon_mode_t mode, size_t* bytes);

/*
 * Build a handle for a fixed parameter set.
 *   shapes:    host array of n shapes (copied).
 *   workspace: device pointer, 1024-byte aligned, ws_bytes >= muon_workspace_size().
 *              It is zero-filled here, on the legacy default stream, and the call
 *              returns once that is done: the handle may be used on any stream at
 *              once.  No earlier work on any stream may still use that memory.  It
 *              must outlive the handle.
 * Uses the current CUDA device, which must be sm_100 (B200).  The handle is
 * bound to that device.
 */
MUON_API muon_status_t muon_create(muon_handle_t* handle, const muon_shape_t* shapes, int n, muon_dtype_t dtype,
                          muon_mode_t mode, void* workspace, size_t ws_bytes);

/*
 * One Muon step for every matrix of the handle, enqueued on `stream`.
 *   W, G, M: host arrays of n device pointers, in the order of the shapes given to
 *            muon_create; matrix i is rows_i x cols_i, row-major, contiguous, of the
 *            handle's dtype.  W and M are updated in place; G is only read.  Any
 *            alignment is accepted; 16-byte aligned rows take the vector path.
 *   hp:      host pointer, read before returning.
 * Returns MUON_ERR_INVALID_ARG for null arrays/pointers or bad hyper-parameters.
 */
MUON_API muon_status_t muon_step(muon_handle_t handle, void* const* W, const void* const* G, void* const* M,
                        const muon_hparams_t* hp, cudaStream_t stream);

/*
 * The orthogonaliser alone: O_i = NS_k(X_i) (normalise, k iterations, orient back),
 * with no momentum and no parameter write.  X and O are host arrays of n device
 * pointers of the handle's dtype and shapes; X is only read.  Only hp->eps, a, b, c
 * and ns_steps are used.
 */
MUON_API muon_status_t muon_orthogonalize(muon_handle_t handle, const void* const* X, void* const* O,
                                 const muon_hparams_t* hp, cudaStream_t stream);

/*
 * `count` equal matrices where and how the caller holds them: element (r, c) of matrix e is at
 * data[e * batch_stride + r * row_stride + c * col_stride], strides in elements and not
 * negative, one of row_stride and col_stride 1 (a matrix stored by rows or by columns; the
 * stride of a dimension of size 1 does not matter).  Slices of fused weights, stacks of heads
 * and transposed storage are views; so is a contiguous matrix.  Rows that start 16-byte
 * aligned take vector accesses.
 */
typedef struct {
  void* data;
  int64_t count, batch_stride, row_stride, col_stride;
  muon_dtype_t dtype;
} muon_view_t;

/*
 * The orthogonaliser on views (MUON_MODE_HALF): O_i = NS_k(X_i) for the matrices of the handle, in
 * order; view j covers its `count` next matrices, which must have one shape (X and O have n views of
 * equal counts, adding up to the handle's matrices).  Each view has its own storage type: bf16,
 * fp16 or fp32.  O_i may be X_i itself (the same view); otherwise an output overlaps no input and no
 * other output (of what would race, equal addresses are refused with MUON_ERR_INVALID_ARG).
 * Only hp->eps, a, b, c and ns_steps are used; muon_set_coefficients overrides a, b, c.
 * Returns MUON_ERR_UNSUPPORTED for a handle of another mode and for views that
 * are stored neither by rows nor by columns.
 */
MUON_API muon_status_t muon_orthogonalize_views(muon_handle_t handle, const muon_view_t* X, const muon_view_t* O,
                                                int n, const muon_hparams_t* hp, cudaStream_t stream);

/*
 * Coefficients of each Newton-Schulz iteration (MUON_MODE_HALF): abc is a host array of
 * steps x 3 floats, iteration t (from 0) of later calls on the handle uses
 * abc[3 t .. 3 t + 2] instead of the hyper-parameters' a, b, c.  A call with more iterations
 * than that is refused with MUON_ERR_INVALID_ARG.  steps = 0 goes back to the hyper-parameters.
 */
MUON_API muon_status_t muon_set_coefficients(muon_handle_t handle, const float* abc, int steps);

/*
 * 8-bit optimizer state.  `count` matrices of rows x cols, back to back: codes holds one byte a value
 * (row-major), scales one fp32 for each MUON_STATE_BLOCK columns of a row, [count][rows]
 * [ceil(cols / MUON_STATE_BLOCK)].  With t the largest magnitude of a block:
 *   INT8  code = x * (127 / t) rounded to an integer, scale = t / 127
 *   E4M3  code = x * (448 / t) rounded to e4m3,       scale = t / 448
 * and code * scale is the value.  E4M3 keeps small values beside large ones (relative steps of
 * 1/16 to 1/8 over a range of 2^15); INT8 is finer (1/127 of t) where a block's values are
 * alike.  A block with t < 2^-100 becomes zeros with scale 0; one that holds an infinity or
 * a NaN gets the scale NaN, so that reading it shows it.  An all-zero state (zero bytes) is zero.
 *
 * Rounding is to nearest even where `seed` is NULL.  Otherwise it is stochastic: up with the
 * probability of the remainder (to 16 bits), by a generator that depends on *seed (read
 * before returning), the matrix's place in the call and the value's place in the matrix only.
 * Give every step another seed, and each of a step's calls (on several handles or ranks) one of its own: equal
 * places of two calls with one seed share their bits.  A captured call repeats the seed it was captured with.
 */
#define MUON_STATE_BLOCK 128
typedef enum { MUON_STATE_INT8 = 0, MUON_STATE_E4M3 = 1 } muon_state_format_t;
typedef struct {
  void* codes;
  float* scales;
  int64_t count, rows, cols;
} muon_state_t;

/*
 * Write n states from views (quantise), and read them back into views (dequantise).  View j has the
 * count and shape of state j and col_stride 1; all views of a call have one type.
 * No handle and no workspace; enqueued on `stream`, with the tensors' device current.  n == 0 is a
 * no-op.  Returns MUON_ERR_INVALID_ARG for null pointers, bad sizes, types or formats,
 * mixed types and overlapping outputs, MUON_ERR_UNSUPPORTED for another col_stride or a matrix of 2^31
 * blocks or more.
 */
MUON_API muon_status_t muon_state_quantize(const muon_view_t* X, const muon_state_t* S, int n,
                                           muon_state_format_t format, const uint32_t* seed, cudaStream_t stream);
MUON_API muon_status_t muon_state_dequantize(const muon_state_t* S, const muon_view_t* X, int n,
                                             muon_state_format_t format, cudaStream_t stream);

/*
 * Momentum and Nesterov blend on 8-bit state, with the Frobenius norms: the first stage of a step,
 * for the handle's matrices in order (any mode).  Per matrix, with m read from the state,
 *   m1 = beta m + (1-beta) g;  u = (1-beta) g + beta m1 if nesterov, else m1
 * in fp32; u is rounded once into U, m1 once into the state.  G and U are views of the handle's type
 * with col_stride 1 (U may be G).  Only hp->beta and nesterov are used.  The norms
 * of u are read with muon_get_norms (where the squares of u leave fp32's range, below 1e-19 or above
 * 1e19, they are those of U as it is stored).
 */
MUON_API muon_status_t muon_momentum_state(muon_handle_t handle, const muon_view_t* G, const muon_state_t* S,
                                           const muon_view_t* U, int n, muon_state_format_t format,
                                           const muon_hparams_t* hp, const uint32_t* seed, cudaStream_t stream);

/*
 * The Muon step on 8-bit momentum (MUON_MODE_HALF): muon_step with M held in S.  W and G are views of the
 * handle's type (G with col_stride 1).  The direction stays in fp32 until it has been normalised
 * (a first pass over G and the state takes the norms, a second one writes).
 */
MUON_API muon_status_t muon_step_state(muon_handle_t handle, const muon_view_t* W, const muon_view_t* G,
                                       const muon_state_t* S, int n, muon_state_format_t format,
                                       const muon_hparams_t* hp, const uint32_t* seed, cudaStream_t stream);

/*
 * AdamW for the parameters that are not matrices: the other half of the hybrid
 * optimizer ("开发者千美元训3.8B模型 击败GPT-2", aiproducthub, 影响 paragraph:
 * Newton-Schulz orthogonalisation for the matrix parameters, AdamW for the rest).
 * The pages print no formula; per element, with t = hp->step >= 1:
 *   m1 = beta1 m + (1-beta1) g;  v1 = beta2 v + (1-beta2) g^2
 *   p1 = (1 - lr wd) p - lr (m1 / (1-beta1^t)) / (sqrt(v1 / (1-beta2^t)) + eps)
 *   P, G: host arrays of n device pointers to tensors of numel[i] elements of
 *         `dtype` (any shape, contiguous); P is updated in place, G only read.
 *   M, V: host arrays of n device pointers to numel[i] fp32 moments each,
 *         updated in place.
 * No handle and no workspace: the call is stateless (the step count is the
 * caller's).  16-byte-aligned tensors take the vector path.  Returns
 * MUON_ERR_INVALID_ARG for null pointers, negative sizes, step < 1, betas
 * outside [0, 1), eps < 0 or non-finite lr/wd; n == 0 is a no-op.
 */
typedef struct {
  float lr, beta1, beta2, eps, weight_decay;
  int32_t step;
} muon_adamw_hparams_t;
MUON_API muon_status_t muon_adamw_step(void* const* P, const void* const* G, float* const* M, float* const* V,
                                       const int64_t* numel, int n, muon_dtype_t dtype,
                                       const muon_adamw_hparams_t* hp, cudaStream_t stream);

/*
 * Copy the n per-matrix Frobenius norms ||U_i||_F of the last step (fp32) into
 * `dst` (host or device memory, n floats), enqueued on `stream`.  Host memory
 * should be pinned for the copy to stay asynchronous.
 */
MUON_API muon_status_t muon_get_norms(muon_handle_t handle, float* dst, cudaStream_t stream);

/*
 * Synchronise `stream`, read the device status word of the handle and clear it (on `stream` too).
 * Returns MUON_OK, MUON_ERR_TIMEOUT or MUON_ERR_DEVICE_STATUS (device fault
 * recorded since the last call), or MUON_ERR_CUDA if the stream reported an error.
 */
MUON_API muon_status_t muon_get_status(muon_handle_t handle, cudaStream_t stream);

/*
 * Failure-detection self-test: enqueue one kernel whose only work is a wait on a
 * shared-memory barrier that nothing signals, bounded by `timeout_ns`
 * (1e3 .. 1e10).  The kernel gives up, records MUON_ERR_TIMEOUT in the status
 * word and returns; muon_get_status() then reports it.  Uses the same bounded
 * wait as the GEMM pipelines.
 */
MUON_API muon_status_t muon_selftest_timeout(muon_handle_t handle, uint64_t timeout_ns, cudaStream_t stream);

/* Release the handle (host memory only; the workspace stays the caller's). */
MUON_API muon_status_t muon_destroy(muon_handle_t handle);

/* Static, human-readable name of a status code. */
MUON_API const char* muon_status_string(muon_status_t status);

/*
 * Plan introspection: the number of shape groups the handle formed, and the
 * number of kernel launches one muon_step with `ns_steps` iterations enqueues
 * (the memset of the arrival counters is not a kernel and is not counted).
 */
MUON_API muon_status_t muon_get_plan(muon_handle_t handle, int ns_steps, int* n_groups, int* launches_per_step);

/*
 * Host-only consistency check of the launch tables muon_step would build for
 * these shapes on a device with num_sms SMs (no device needed): the persistent
 * momentum/norm kernel's tile ranges and partial-sum slots, and the single-launch
 * schedule's tile list for ns_steps iterations (every stage of every matrix
 * covered once, stages listed before the tiles that wait for them, wait targets
 * equal to the stages' tile counts), with and without the fused parameter
 * write.  *problems receives the number of inconsistencies (0 when sound).  For
 * tests and tools.
 */
MUON_API muon_status_t muon_check_plan(const muon_shape_t* shapes, int n, int ns_steps, int num_sms,
                                       int64_t* problems);

/*
 * How the k Newton-Schulz iterations of a MUON_MODE_FAST or MUON_MODE_HALF handle are launched (in HALF:
 * of the shape groups that do not run on chip; the conditions below are about those).
 *   MUON_SCHEDULE_STAGED  one tensor-core launch per stage and iteration (3 k
 *                         launches: Gram, polynomial, update), each over every
 *                         matrix of the handle.
 *   MUON_SCHEDULE_FUSED   all 3 k stages in one persistent launch: the tiles of
 *                         every stage form one list, and a tile waits (on the
 *                         device, bounded) only until the stage it reads is
 *                         complete for its own matrix, so the stages of different
 *                         matrices overlap and no launch boundary drains the GPU.
 *                         Same arithmetic and rounding as STAGED (results are
 *                         bitwise equal).  Needs at most 6 distinct shape groups.
 *                         Launches of several handles, and other work, may share
 *                         the GPU: the tiles go to the CTAs that got an SM.
 *   MUON_SCHEDULE_SPLIT   the tiles of FUSED, one launch per stage (3 k launches):
 *                         separates the single-launch kernel's tile machinery
 *                         from its scheduling, for measurements.
 *   MUON_SCHEDULE_AUTO    (default) FAST: FUSED when every shape group's smaller
 *                         dimension is at most 768 (there it measured within 1 %
 *                         of STAGED with one launch per step instead of 3 k),
 *                         else STAGED.  HALF: FUSED up to eight 256 x 256 Update
 *                         tiles for each pair of SMs, else STAGED.
 * The small-matrix kernel (MUON_KERNEL_NS_SMALL) keeps precedence when its
 * conditions hold; FP32_REF handles always run staged.  Returns
 * MUON_ERR_UNSUPPORTED if FUSED is asked of a handle that cannot run it.
 * The setting applies to later calls; it must not change while a captured graph
 * of the handle is replayed.
 */
#define MUON_SCHEDULE_AUTO 0
#define MUON_SCHEDULE_STAGED 1
#define MUON_SCHEDULE_FUSED 2
#define MUON_SCHEDULE_SPLIT 3
MUON_API muon_status_t muon_set_schedule(muon_handle_t handle, int schedule);

/*
 * Momentum, Nesterov blend and Frobenius norm of ONE matrix, with no workspace.
 * The pages have no counterpart for this entry point: it exists for callers that
 * cannot give this library device memory (a framework whose allocator must own
 * every device allocation, a fixed memory pool, code that may not call
 * cudaMalloc).  It computes, for the rows x cols row-major matrix of `dtype`,
 *   M <- beta*M + (1-beta)*G   (in place),
 *   U <- (1-beta)*G + beta*M   if nesterov, else U <- M   (U: same shape/dtype),
 *   *norm <- ||U||_F           (fp32; `norm` is a device pointer to one float),
 * the same arithmetic as the first stage of muon_step (U in the caller's layout,
 * not transposed).  The norm's reduction scratch is a fixed array of device
 * memory inside libmuon.so (about 16 KB, held by every GPU that loads the
 * library until the process exits); the call allocates nothing.
 *   - rows * cols may be at most MUON_STATIC_MAX_ELEMENTS, else
 *     MUON_ERR_UNSUPPORTED is returned and nothing is enqueued.
 *   - The first call on a device (with that device current) looks up the
 *     array's device address; make it before capturing any stream.  A first
 *     call on a stream that is being captured returns MUON_ERR_UNSUPPORTED
 *     without touching the capture.
 *   - All calls share the array.  Calls in sequence on one stream are
 *     independent (the arrival counter is cleared at the start of each call);
 *     calls that overlap on the GPU race and give wrong norms.
 */
#define MUON_STATIC_MAX_ELEMENTS (1ll << 28)
MUON_API muon_status_t muon_momentum_norm_static(const void* G, void* M, void* U, int64_t rows, int64_t cols,
                                                 muon_dtype_t dtype, float beta, int32_t nesterov, float* norm,
                                                 cudaStream_t stream);

/*
 * Workspace introspection, for tests and tools.  muon_get_matrix_slot gives the
 * shape group of matrix i and its slot inside the group's batched buffers;
 * muon_get_group_buffers gives a group's padded oriented shape (mp x np, both
 * multiples of 256), its matrix count and the device addresses of its buffers
 * inside the workspace: X0 and X1 ([count][mp][np]) and A and B
 * ([count][mp][mp]), elements bf16 in FAST mode, fp32 in FP32_REF mode and fp16 in HALF mode
 * (there X0 is the normalised X times 2^12, and the addresses of a group that runs on chip are NULL).
 * After muon_orthogonalize/muon_step with k iterations, X0 holds U (oriented,
 * unnormalised), A and B hold the last iteration's Gram and polynomial
 * matrices, and X(k mod 2) the final iterate.  Any output pointer may be NULL.
 */
MUON_API muon_status_t muon_get_matrix_slot(muon_handle_t handle, int i, int* group, int* slot);
MUON_API muon_status_t muon_get_group_buffers(muon_handle_t handle, int group, int* mp, int* np, int* count,
                                              void** x0, void** x1, void** a, void** b);

/*
 * Kernel tracing with CUDA events (no device memory).  After
 * muon_profile_begin(h, max_steps), each of the next max_steps calls of
 * muon_step / muon_orthogonalize records one event before its first kernel and
 * one after every kernel, on the caller's stream.  muon_profile_end()
 * synchronises those events, writes for each kernel kind k (MUON_KERNEL_*) the
 * summed device milliseconds ms[k] and the number of launches launches[k]
 * (arrays of n_kinds entries, host memory), destroys the events and stops
 * recording.  The time of a kernel is the gap between the events around it.
 */
#define MUON_KERNEL_MOMENTUM_NORM 0
#define MUON_KERNEL_GRAM 1
#define MUON_KERNEL_POLY 2
#define MUON_KERNEL_UPDATE 3
#define MUON_KERNEL_WRITE 4
#define MUON_KERNEL_SGEMM 5
#define MUON_KERNEL_NS_SMALL 6 /* all iterations of a set of matrices of at most 256 x 256 */
#define MUON_KERNEL_NS_FUSED 7 /* all iterations of a set in one launch (MUON_SCHEDULE_FUSED) */
#define MUON_KERNEL_KINDS 8
MUON_API muon_status_t muon_profile_begin(muon_handle_t handle, int max_steps);
MUON_API muon_status_t muon_profile_end(muon_handle_t handle, double* ms, int* launches, int n_kinds);

#ifdef __cplusplus
}
#endif

#endif /* MUON_H_ */
