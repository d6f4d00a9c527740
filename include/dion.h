/*
 * libdion — one Dion / Orth-Dion optimizer step on an AMD MI355X (gfx950).
 *
 * The step is the one written out on the "Orth-Dion" documentation page
 * (junaidaliop.github.io, zij/math/orthdion): its equation block and the
 * symbol list below it.  For a weight matrix X (m x n) with gradient G,
 * error-feedback residual R (both m x n) and warm start V (n x r):
 *
 *   M    = G + R                       buffer
 *   U    = orth(M V)                   one warm-started power-iteration step
 *   W    = M^T U                       right factor
 *   Vbar = orth(W)                     Orth-Dion
 *        = W diag(1 / ||w_j||_2)       Dion (the page's closing remark: column
 *                                      normalization in place of orth)
 *   X   <- X - eta U Vbar^T
 *   R   <- beta (M - U W^T)            (U^T M = W^T, so W is reused)
 *   V   <- Vbar                        warm start of the next step
 *
 * orth(A) is the Q factor of the thin QR factorization A = Q T whose upper
 * triangular T has a positive diagonal (the symbol list defines orth as the
 * QR orthonormalization of the column space; the positive diagonal makes Q
 * unique for a full-rank A).  The library computes it by CholeskyQR: a
 * float64 Gram matrix (assembled from exact int8 digit products on the
 * matrix cores by default, see DION_GRAM_F64), a blocked float64 Cholesky
 * factorization S = T^T T that also yields T^{-T}, and the product
 * A T^{-1} on the matrix cores.  The pivots tell how well-conditioned A is
 * (pivot j over S_jj is about 1 / kappa^2 at worst):
 *   - kappa below about 1e3 (every pivot ratio >= 1e-6): that one pass;
 *   - up to about 1e4: a second pass on the result (CholeskyQR2) with a
 *     float64 Gram matrix and float64 products;
 *   - beyond that, or a failed pivot: the first pass is redone with a
 *     diagonal shift on a float64 Gram matrix (shifted CholeskyQR), then
 *     the second pass follows.
 * The choice is made per matrix on the device.  A factor that is rank-
 * deficient to float32 accuracy (the second pass finds a pivot ratio below
 * 2 r 2^-48) is a breakdown (see below).
 *
 * Conventions for every entry point:
 *   - All functions are extern "C"; no C++ exception crosses the boundary.
 *   - Matrices are dense row-major (C order) with no padding: element (i, j)
 *     of an a x b matrix is at p[i * b + j].  X, R, V are float32; G is
 *     float32 or bfloat16 (raw 16-bit patterns), chosen by g_dtype.
 *   - All pointers passed as matrices or workspace are DEVICE pointers on the
 *     current HIP device.  The caller owns them.  X, R and V are updated in
 *     place; G is only read.  X, G, R, V and the workspace must not overlap.
 *     They need natural alignment (4 bytes; 2 for bfloat16 G); 16-byte
 *     aligned pointers with a column count divisible by 4 take the vector
 *     load path.
 *   - stream is a hipStream_t (NULL = the default stream).  Work is only
 *     enqueued: the calls return before the GPU finishes and never
 *     synchronize the host, except dion_status, dion_plan_destroy and
 *     dion_plan_timing_enable / _read, which wait for work they must read
 *     or free.  Buffers must stay valid until the enqueued work completes.
 *   - Argument errors are reported synchronously, before any HIP call is
 *     made, and leave every buffer untouched.
 *   - A numerical breakdown (orth of a factor that is rank-deficient to
 *     float32 accuracy or not finite; a zero or non-finite column norm for
 *     Dion) can only be seen on the device.  It is recorded in a status
 *     word inside the workspace, and every later kernel of that matrix skips
 *     its writes, so X, R and V of that matrix keep their previous contents
 *     bit for bit.  Read it with dion_status.
 */
#ifndef LIBDION_DION_H_
#define LIBDION_DION_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define DION_OK               0
#define DION_ERR_INVALID_ARG (-1)  /* null pointer, bad size, rank, variant, dtype, non-finite eta/beta */
#define DION_ERR_WORKSPACE   (-2)  /* workspace missing or smaller than required */
#define DION_ERR_HIP         (-3)  /* a HIP runtime call or kernel launch failed */
#define DION_ERR_BREAKDOWN   (-4)  /* (dion_status only) numerical breakdown on the device */

/* Right-factor rule: equation 4 of the Orth-Dion page, or Dion's column
 * normalization. */
#define DION_VARIANT_DION 0
#define DION_VARIANT_ORTH 1
#define DION_VARIANT_MASK 0xff

/* Arithmetic of the three m x n x r products (P = M V, W = M^T U and the
 * X / R update), OR-ed into the `variant` argument of every entry point.
 * DION_MATH_F32 (default): float32 MFMA products, float32 accumulation.
 * DION_MATH_BF16X3: each float32 operand x is split into bfloat16
 *   hi = bf16(x) and lo = bf16(x - hi), and a product is taken as
 *   hi*hi + hi*lo + lo*hi on the bfloat16 matrix cores with float32
 *   accumulation: relative product error up to 2^-16 instead of 2^-24, at
 *   about five times the float32 matrix rate.  orth() (the Gram matrix
 *   below, the triangular product in float32) is unaffected. */
#define DION_MATH_F32     0x000
#define DION_MATH_BF16X3  0x100
#define DION_MATH_MASK    0x100

/* Gram matrix S = Q^T Q of orth()'s CholeskyQR pass (orth() of equations 2
 * and 4 of the Orth-Dion page), OR-ed into `variant` like the math mode.
 * Default: each float32 column q_j of Q is scaled by a power of two into
 *   (-1, 1) and written as five signed base-128 digits (int8); S is
 *   assembled in float64 from the 15 leading digit products, each summed
 *   exactly in int32 on the int8 matrix cores.  Each product q_ik q_jk
 *   enters S with an error below 2^-30 max|q_i| max|q_j| (the digits'
 *   remainder and the dropped digit products); over many rows these errors
 *   add like independent roundings (measured: Gram entries within 2e-10 of
 *   sqrt(S_ii S_jj) of the float64 Gram).  A non-finite entry of Q makes
 *   its row and column of S NaN, a breakdown of the factorization.
 * DION_GRAM_F64: float32 products summed in float64 on the float64 matrix
 *   cores (products exact, float64 rounding only). */
#define DION_GRAM_F64     0x400

/* Schedule of small matrices.  By default a matrix with r <= 16 whose
 * step is small (factors P, W and V within 64 KB once their columns are
 * padded to 8 or 16, and m n r <= 2^21) takes the whole step in one
 * workgroup of one launch: float32 products, float64 Gram matrix and
 * Cholesky, float64 triangular products (the math mode does not apply to
 * it).  DION_SCHED_GROUPED, OR-ed into `variant`, sends every matrix
 * through the grouped multi-launch schedule instead.  Sharded plans always
 * use the grouped schedule. */
#define DION_SCHED_GROUPED 0x800

/* Row-sharded step (FSDP layout; the sharded setting the Dion and
 * Orth-Dion abstracts motivate).  OR DION_SHARDED into the variant of
 * dion_plan_create for a plan whose matrices are the local row shards of
 * the global matrices: matrix i is rows [a_i, a_i + m_i) of some global
 * X, G, R (m_i x n), and every shard of one global matrix holds its own
 * copy of the same V (n x r).  dion_plan_shard_stage then runs the step in
 * three stages; between them the caller sums one exchange buffer over all
 * shards of each global matrix (an all-reduce across GPUs; with a single
 * shard there is nothing to do) and writes the sum back into every shard's
 * buffer:
 *   stage 0: P_i = M_i V and the local Gram partial P_i^T P_i
 *            -> exchange DION_SHARD_GRAM: float64, rp x rp row-major
 *               (rp = r rounded up to 64); stage 1 reads only the upper
 *               triangle of its leading r x r block
 *   stage 1: T from the summed Gram matrix, U_i = P_i T^{-1},
 *            W_i = M_i^T U_i (one CholeskyQR pass: a further pass would
 *            need another exchange, so a pivot ratio below 1e-6 is a
 *            breakdown here; orth(W) in stage 2 takes every pass it needs)
 *            -> exchange DION_SHARD_W: float32, n x r row-major
 *   stage 2: Vbar from the summed W (computed identically on every shard),
 *            X_i and R_i updated, Vbar written into the shard's V.
 * Summed this way the shards' results equal one step on the global
 * matrices.  dion_plan_shard_buffer gives the byte offset (from the
 * workspace base) and size of exchange buffer `which` (DION_SHARD_*) of
 * matrix `index` (position in the plan's list).  Stage calls follow the
 * order 0, 1, 2 on one workspace and stream; the buffers are valid from
 * the end of the stage that writes them to the start of the next stage.
 * dion_plan_step also runs a sharded plan: all three stages without
 * exchange, i.e. each shard as a matrix of its own.  dion_step and
 * dion_step_batched reject DION_SHARDED (DION_ERR_INVALID_ARG).  Errors:
 * DION_ERR_INVALID_ARG for a null plan, a plan created without
 * DION_SHARDED, a stage outside 0..2, which outside DION_SHARD_*, an index
 * outside the list or a null output pointer; otherwise as dion_plan_step.
 * A shard may have fewer rows than r (only r <= n is required of it); the
 * global matrix needs at least r rows for its Gram matrix to be definite. */
#define DION_SHARDED      0x200
#define DION_SHARD_GRAM   0
#define DION_SHARD_W      1

/* Element type of G. */
#define DION_DTYPE_F32  0
#define DION_DTYPE_BF16 1

/* Per-matrix breakdown flags reported by dion_status (0 = step applied). */
#define DION_STATUS_ORTH_P   1   /* orth(M V) failed */
#define DION_STATUS_ORTH_W   2   /* orth(W) failed (Orth-Dion) */
#define DION_STATUS_COLNORM  4   /* zero or non-finite column norm (Dion) */

/* Upper bounds accepted by the library. */
#define DION_MAX_DIM   (1 << 20)      /* m, n */
#define DION_MAX_RANK  4096           /* r */

/* One matrix of a grouped step.  Device pointers, row-major, see above. */
typedef struct dion_matrix {
    float*       X;   /* m x n, updated in place */
    const void*  G;   /* m x n, float32 or bfloat16 per g_dtype, read only */
    float*       R;   /* m x n, updated in place */
    float*       V;   /* n x r, warm start in, Vbar out */
    int64_t      m, n, r;
} dion_matrix;

/* Opaque handle for a grouped step over a fixed list of matrices. */
typedef struct dion_plan dion_plan;

/* Library version as major * 10000 + minor * 100 + patch. */
int dion_version(void);

/* Static string for a return code (never NULL). */
const char* dion_error_string(int code);

/* Workspace bytes one dion_step call on an m x n matrix of rank r needs.
 * Returns 0 when the arguments are invalid. */
size_t dion_workspace_size(int64_t m, int64_t n, int64_t r, int variant, int g_dtype);

/* One step on one matrix (the equations at the top of this header).
 *   X, G, R, V: device pointers (see conventions); m, n >= 1; 1 <= r <= min(m, n).
 *   eta: learning rate, beta: error-feedback coefficient (finite floats).
 *   variant: DION_VARIANT_*; g_dtype: DION_DTYPE_*.
 *   workspace: device buffer of at least dion_workspace_size(...) bytes,
 *   16-byte aligned, owned by the caller; its contents need not be preserved
 *   between calls except for the status word read by dion_status.
 * Returns DION_OK once the work is enqueued, or an error code (nothing
 * enqueued for argument errors). */
int dion_step(float* X, const void* G, float* R, float* V,
              int64_t m, int64_t n, int64_t r, float eta, float beta,
              int variant, int g_dtype,
              void* workspace, size_t workspace_bytes, void* stream);

/* dion_step for callers that cannot allocate device memory (code under HIP
 * graph capture, serving loops or harnesses that forbid allocation): the
 * same step with the same kernels, its workspace taken from a scratch array
 * that the library holds on each GPU (32 MiB, kept until the process ends)
 * instead of a caller buffer.  No device memory is allocated or freed.
 * Shapes whose workspace (dion_workspace_size) exceeds 32 MiB are rejected
 * with DION_ERR_WORKSPACE before any HIP call (for example 1024 x 1024 at
 * rank 256, or 768 x 3072 at rank 192, fit; 2048 x 2048 at rank 512 does
 * not).  All calls on one GPU share its scratch, so calls that overlap on
 * one GPU (other streams, other threads) race; calls in stream order do
 * not.  status_out (optional, a device pointer to one int) receives the
 * matrix's status word when the step ends: its bits 0-7 are the
 * DION_STATUS_* flags (0: the step was applied); higher bits are internal.
 * Other arguments and errors as dion_step. */
int dion_step_noalloc(float* X, const void* G, float* R, float* V,
                      int64_t m, int64_t n, int64_t r, float eta, float beta,
                      int variant, int g_dtype, int* status_out, void* stream);

/* Grouped step: the same update applied to each matrix of a list (for
 * example all weight matrices of a model) with a handful of kernel launches
 * for the whole list.  The pages apply the step to every weight matrix
 * independently (Orth-Dion page, equation block, per matrix X); the nearest
 * thing they describe to running many of them together is the Dion3
 * abstract's megabatching.  Matrices may have different shapes.  Equivalent
 * to a dion_step call per matrix.  The matrix list is copied; the call
 * keeps an internal cache of plans keyed by the list, so repeating the same
 * list costs no host-side setup (a plan evicted from the cache is freed
 * once its last copy has completed, without waiting for it). */
size_t dion_workspace_size_batched(const dion_matrix* mats, int count,
                                   int variant, int g_dtype);
int dion_step_batched(const dion_matrix* mats, int count, float eta, float beta,
                      int variant, int g_dtype,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Explicit plan for a grouped step (what dion_step_batched caches).
 * dion_plan_create validates the list and builds the schedule on the host;
 * it allocates pinned host memory for the matrix table (no device memory).
 * dion_plan_step enqueues one grouped step: an asynchronous copy of the
 * table into the workspace, then the kernels.  dion_plan_destroy waits for
 * the last table copy of this plan to finish, then frees it. */
int    dion_plan_create(const dion_matrix* mats, int count, int variant,
                        int g_dtype, dion_plan** plan_out);
size_t dion_plan_workspace_size(const dion_plan* plan);
int    dion_plan_count(const dion_plan* plan);
int    dion_plan_step(dion_plan* plan, float eta, float beta,
                      void* workspace, size_t workspace_bytes, void* stream);
void   dion_plan_destroy(dion_plan* plan);

int dion_plan_shard_stage(dion_plan* plan, int stage, float eta, float beta,
                          void* workspace, size_t workspace_bytes, void* stream);
int dion_plan_shard_buffer(const dion_plan* plan, int which, int index,
                           size_t* offset, size_t* bytes);

/* Inspection of a plan's intermediate factors.  After a step of `plan` has
 * completed on the stream, the workspace holds, for matrix `index` (its
 * position in the plan's list) unless it broke down:
 *   DION_BUF_P  P = M V                 float32, m x r row-major
 *   DION_BUF_U  U = orth(P)             float32, m x r row-major
 *   DION_BUF_W  W = M^T U               float32, n x r row-major
 * dion_plan_buffer gives the byte offset from the workspace base and the
 * size of one of them.  They stay valid until the next step on that
 * workspace.  Errors: DION_ERR_INVALID_ARG for a null plan or output
 * pointer, `which` outside DION_BUF_* or `index` outside the list. */
#define DION_BUF_W    1   /* the same value as DION_SHARD_W */
#define DION_BUF_P    2
#define DION_BUF_U    3
int dion_plan_buffer(const dion_plan* plan, int which, int index,
                     size_t* offset, size_t* bytes);

/* Phase timing, for measurement.  A step runs five phases, in order:
 *   0  P = M V            1  U = orth(P)          2  W = M^T U
 *   3  Vbar (orth(W) or column normalization; with split-bfloat16 products
 *      also the bfloat16 planes of U, W and Vbar the update reads)
 *   4  X and R update (the update kernel alone)
 * dion_plan_timing_enable(plan, max_steps) makes the next max_steps calls of
 * dion_plan_step record a HIP event at every phase boundary on the step's
 * stream (creating the events now; 0 disables and frees them).
 * dion_plan_timing_read waits for the last recorded event, writes the
 * summed milliseconds of each phase over the recorded steps into
 * ms_per_phase[DION_PHASES] and the step count into *steps, and starts a
 * new recording window. */
#define DION_PHASES 5
int dion_plan_timing_enable(dion_plan* plan, int max_steps);
int dion_plan_timing_read(dion_plan* plan, double* ms_per_phase, int* steps);

/* Breakdown check: waits for `stream`, then reads the status words of the
 * last step enqueued on `workspace` (count = 1 for dion_step, the list
 * length for a grouped step).  per_matrix (optional, count ints) receives
 * each matrix's DION_STATUS_* flags, in the caller's list order.
 * Returns DION_OK, DION_ERR_BREAKDOWN if any matrix broke down, or an
 * argument / HIP error.  The workspace does not record how many matrices
 * the last step had, so the caller passes `count`; a grouped step can
 * break down in some matrices only, so the flags come per matrix rather
 * than as one code. */
int dion_status(const void* workspace, int count, void* stream, int* per_matrix);

/* ---------------------------------------------------------------------------
 * Orthogonalization by Newton-Schulz products, and the Muon step.
 *
 * For an m x n matrix G, on its smaller side (A is p x p, p = min(m, n)):
 *   X = G / ||G||_F, then for each iteration k:
 *   X <- a_k X + (b_k A + c_k A^2) X,   A = X X^T
 *   O = the last X
 * which moves every singular value s by s <- a s + b s^3 + c s^5 and keeps
 * the singular vectors.  coeffs holds steps triples (a, b, c); a triple with
 * c = 0 is a cubic iteration and takes two products instead of three.  The
 * usual five quintic iterations take (3.4445, -4.7750, 2.0315) each; the
 * textbook cubic is (1.5, -0.5, 0).  1 <= steps <= 32.  Coefficients under
 * which a singular value in [0, 1] can grow past 64 are rejected.
 *
 * math: DION_MATH_F32 keeps float32 accuracy (every factor as two float16
 *   planes, 22 bits, three matrix products per product); DION_MATH_F16 takes
 *   one float16 product per product (factors rounded to 11 bits between
 *   products, float32 accumulation): about 1.2e-3 relative error after five
 *   quintic iterations of an N(0, 1) matrix, below bfloat16's own rounding of
 *   the result, growing for matrices whose singular values fall off steeply.
 *   A matrix whose smaller side is at most 128 keeps float32 accuracy in both
 *   (its roundings would average over too few singular values), one of at most
 *   16 rows or columns is computed in plain float32.  Entries are
 *   held relative to the largest singular value that the coefficients allow:
 *   coefficients that shrink everything far below it lose accuracy.
 *
 * A zero matrix has O = 0.  A matrix with a non-finite entry (or, for the
 * step, a non-finite momentum) sets DION_STATUS_NONFINITE in its status word
 * (dion_status) and leaves O, or X and M, as they were.  The conventions at
 * the top of this header hold, with these differences: G and O have row
 * pitches ldg, ldo >= n (elements, < 2^31) and may be column blocks of one
 * buffer, of one pitch; 1 <= m, n <= DION_MAX_DIM with m n < 2^31 and any order;
 * a list holds at most DION_MAX_LIST matrices.  The list is read before the
 * call returns.  The same call gives the same bits; a matrix's last bits may
 * depend on the other matrices of the list (long sums are cut to fill the
 * chip). */
#define DION_MATH_F16     0x1000
#define DION_STATUS_NONFINITE 8  /* orthogonalize, muon_step: non-finite input */
#define DION_MAX_LIST 65536

typedef struct dion_ns_matrix {
  const void* G;        /* m x n, float32 or bfloat16 per g_dtype, read only */
  void*       O;        /* m x n, float32 or bfloat16 per o_dtype */
  int64_t     m, n;
  int64_t     ldg, ldo; /* row pitches in elements */
} dion_ns_matrix;

size_t dion_orthogonalize_workspace_size(const dion_ns_matrix* mats, int count, int math);
int dion_orthogonalize_batched(const dion_ns_matrix* mats, int count,
                               const float* coeffs, int steps, int math,
                               int g_dtype, int o_dtype,
                               void* workspace, size_t workspace_bytes, void* stream);
int dion_orthogonalize(const void* G, int64_t ldg, void* O, int64_t ldo,
                       int64_t m, int64_t n, const float* coeffs, int steps, int math,
                       int g_dtype, int o_dtype,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Muon step on dense row-major X, M (float32) and G (float32 or bfloat16):
 *   M <- mu M + G
 *   D  = G + mu M (nesterov != 0) or M
 *   X <- (1 - lr weight_decay) X - lr scale O,   O = orthogonalize(D)
 * X and M are updated in place.  scale is the caller's per-matrix factor
 * (for example sqrt(max(1, m / n))); lr scale and 1 - lr weight_decay have to be
 * finite in float32. */
typedef struct dion_muon_matrix {
  float*      X;        /* m x n, updated in place */
  const void* G;        /* m x n, read only */
  float*      M;        /* m x n momentum, updated in place */
  int64_t     m, n;
  float       scale;
} dion_muon_matrix;

size_t dion_muon_workspace_size(const dion_muon_matrix* mats, int count, int math);
int dion_muon_step_batched(const dion_muon_matrix* mats, int count, float lr, float momentum,
                           int nesterov, float weight_decay, const float* coeffs, int steps,
                           int math, int g_dtype,
                           void* workspace, size_t workspace_bytes, void* stream);
int dion_muon_step(float* X, const void* G, float* M, int64_t m, int64_t n, float scale,
                   float lr, float momentum, int nesterov, float weight_decay,
                   const float* coeffs, int steps, int math, int g_dtype,
                   void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Linear layer: the products around a weight matrix that the steps above
 * train.  x is t x k (tokens by inputs), W n x k:
 *   forward:   z = x W^T + bias;  y = act(z) + residual
 *   backward:  dz = dy act'(z);  dx = dz W;  dW = dz^T x;  db = sum_t dz
 * (the residual's gradient is dy itself).  dW is the G that a step reads.
 *
 * Every tensor has `dtype` (float32 or bfloat16) except bias and db, which
 * are float32, and a row pitch in elements (>= its columns, <= 2^30); elements
 * in their natural alignment, n, k <= DION_MAX_DIM and 0 <= t <= 2^24 (t = 0: dW
 * and db are zero).  bfloat16 products are exact and summed in float32; act,
 * bias and residual are applied in float32 and the result is rounded once;
 * backward of bfloat16 with an activation rounds dz to bfloat16 before the two
 * products (to 16 bits with at most 64 tokens).  float32 products are taken as
 * six bfloat16 products of three-way split operands (24 bits, errors of
 * float32's order; with more than 8 tokens, and in the backward pass, a value
 * below 2^-110 is taken to within 2^-134); a non-finite operand makes the
 * outputs it reaches non-finite, not always with the sign float32 would give.
 *
 * Forward reads x, w, bias (or NULL), residual (or NULL; y itself is allowed)
 * and writes y and, when z is not NULL, z.  Backward reads dy, z (only with
 * an activation), x (for dw) and w (for dx) and writes those of dx, dw and db
 * that are not NULL; with accumulate != 0, dw and db are added to.  Outputs
 * share no element with anything else (column blocks of one buffer, of one
 * pitch, are apart).  Sums are taken in a fixed order: the same call gives
 * the same bits.  Size queries return 0 for invalid arguments; errors as for
 * the calls above. */
#define DION_ACT_NONE  0
#define DION_ACT_RELU  1
#define DION_ACT_RELU2 2   /* max(z, 0)^2 */
#define DION_ACT_GELU  3   /* z Phi(z), Phi the normal distribution function */
#define DION_ACT_SILU  4   /* z / (1 + exp(-z)) */

typedef struct dion_linear {
  int64_t      t, n, k;
  const void*  x;         int64_t ldx;     /* t x k */
  const void*  w;         int64_t ldw;     /* n x k */
  const float* bias;                       /* n */
  const void*  residual;  int64_t ldr;     /* t x n */
  void*        y;         int64_t ldy;     /* t x n */
  void*        z;         int64_t ldz;     /* t x n */
  const void*  dy;        int64_t lddy;    /* t x n */
  void*        dx;        int64_t lddx;    /* t x k */
  void*        dw;        int64_t lddw;    /* n x k */
  float*       db;                         /* n */
  int          act;                        /* DION_ACT_* */
  int          dtype;                      /* DION_DTYPE_* */
  int          accumulate;
} dion_linear;

size_t dion_linear_forward_workspace_size(const dion_linear* l);
int dion_linear_forward(const dion_linear* l, void* workspace, size_t workspace_bytes, void* stream);
size_t dion_linear_backward_workspace_size(const dion_linear* l);
int dion_linear_backward(const dion_linear* l, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Softmax cross entropy of an output head: the product of the hidden states
 * with the head's weight, the loss and its gradients, without keeping the
 * logits.  x is t x k (tokens by inputs), W n x k (n: the vocabulary), y the
 * targets, e label_smoothing, zc z_loss:
 *   forward:   z = x W^T;  lse = log sum_j exp z_j
 *              loss = lse - (1 - e) z_y - e mean_j z_j + zc lse^2
 *   backward:  dz_j = dloss ((1 + 2 zc lse) exp(z_j - lse) - (1 - e) [j = y]
 *                            - e / n)
 *              dx = dz W;  dW = dz^T x
 * per token; dloss is the loss's gradient per token (1 over their number for a
 * mean, say).  A row whose target is ignore_index has loss 0 and dz 0 whatever
 * its logits are (its x still meets that zero in dW: a non-finite x there makes
 * dW NaN); any other target outside 0 .. n - 1 makes its row's loss, and what
 * its dz reaches, NaN.  dW is a G for the steps above.
 *
 * x, w, dx, dw have `dtype` (float32 or bfloat16) and a row pitch in elements
 * (>= k, <= 2^30); target is int64, loss, lse and dloss float32, t contiguous
 * elements each; elements in their natural alignment, n, k <= DION_MAX_DIM,
 * 0 <= t <= 2^24 (t = 0: dW is zero), 0 <= e <= 1.  Products are taken as the
 * linear layer takes them (bfloat16 exact, float32 as six bfloat16 products),
 * sums in float32; dz is rounded to bfloat16 before its two products (to 16
 * bits with at most 64 tokens, to 24 in float32) and computed a piece of the
 * vocabulary at a time.
 *
 * The backward's workspace is at most 256 MiB, or 256 columns of dz (2 bytes per
 * token in bfloat16, 4 in float32) where those are more (from 2^19 and 2^18 tokens
 * on); 200 MiB of products' partial sums; and in bfloat16 t x k float32 where there
 * are several pieces, and copies of operands that the tiles cannot read in place,
 * x and a piece of W (256 MiB, or 256 rows).  With few tokens (64 in bfloat16, 32 in
 * float32) it is at most 320 MiB and 1 KiB per input.  The forward's is at most an
 * eighth of a byte per logit (one and a half times that with label smoothing; few
 * tokens half a byte, of 16384 words at most) and 64 bytes per token, 70 MiB of
 * partial sums, and such copies.
 *
 * Forward reads x, w, target and writes those of loss and lse that are not
 * NULL.  Backward reads x, w, target, lse (forward's) and dloss and writes
 * those of dx and dw that are not NULL; with accumulate != 0, dw is added to.
 * Outputs share no element with anything else.  Sums are taken in a fixed
 * order: the same call gives the same bits.  Size queries return 0 for invalid
 * arguments; errors as for the calls above. */
typedef struct dion_cross_entropy {
  int64_t        t, n, k;
  const void*    x;         int64_t ldx;   /* t x k */
  const void*    w;         int64_t ldw;   /* n x k */
  const int64_t* target;                   /* t */
  float*         loss;                     /* t */
  float*         lse;                      /* t */
  const float*   dloss;                    /* t */
  void*          dx;        int64_t lddx;  /* t x k */
  void*          dw;        int64_t lddw;  /* n x k */
  int64_t        ignore_index;
  float          label_smoothing, z_loss;
  int            dtype;                    /* DION_DTYPE_* */
  int            accumulate;
} dion_cross_entropy;

size_t dion_cross_entropy_forward_workspace_size(const dion_cross_entropy* a);
int dion_cross_entropy_forward(const dion_cross_entropy* a, void* workspace, size_t workspace_bytes,
                               void* stream);
size_t dion_cross_entropy_backward_workspace_size(const dion_cross_entropy* a);
int dion_cross_entropy_backward(const dion_cross_entropy* a, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ---------------------------------------------------------------------------
 * AdamW step for the tensors that the matrix steps above leave alone
 * (embeddings, output heads, norms, biases): for each tensor of n elements,
 * in any order, with g = c G and step t >= 1,
 *   m <- beta1 m + (1 - beta1) g
 *   v <- beta2 v + (1 - beta2) g^2
 *   X <- (1 - lr weight_decay) X
 *        - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * c = *grad_scale, one float32 on the device (a clipping factor or the inverse
 * of a loss scale, say), or 1 where grad_scale is NULL.  A c that is not
 * finite leaves every tensor as it was.
 *
 * state_bits: the moments' form.
 *   DION_STATE_F32   M and V hold m and v in float32; S is not used.
 *   DION_STATE_8BIT  M and V hold m and sqrt(v), one byte per element, in
 *     blocks of DION_ADAMW_BLOCK consecutive elements: an e4m3 value (4 bits of
 *     exponent, 3 of mantissa, no infinities) times the block's scale, a power
 *     of two 2^(b - 127).  S holds the bytes b: first M's, one per block (the
 *     last block may be short), then V's.  All zero is the state before the
 *     first step.  X is stepped with the new moments before they are rounded.
 *     b is the exponent byte of the block's largest magnitude less 7, at
 *     least 1, and a scaled magnitude a < 256 is rounded to floor(a / ulp + u)
 *     ulp, ulp = 2^(max(floor(log2 a), -6) - 3), whose mean over u in [0, 1) is
 *     a: moments move by far less than an ulp per step.  A nonzero sqrt(v) is
 *     never rounded to zero (a moment without its v would be divided by eps).
 *     u comes from the caller's seed, which should differ from step to step,
 *     and the element's index i in its tensor (mod 2^32):
 *       h = (i + 0x632be5ab seed) 0x9e3779b1;  h = (h ^ h / 2^15) 0x85ebca77;
 *       h = h ^ h / 2^13;  u = h mod 2^16 (M), h / 2^16 (V), over 2^16
 *     A block with a new m or v that is not finite becomes NaN as a whole.
 *
 * Everything else that is not finite reaches the elements it belongs to.
 * Tensors of a list share no memory; X, M, V, S and G of one do not overlap, and
 * X, M, V and S do not hold grad_scale.
 * Pointers in their elements' alignment (16 bytes are faster), 0 <= n <= 2^33
 * (n = 0: pointers are not looked at), float32 X, G of one type for the list, at
 * most DION_MAX_LIST tensors.  0 <= beta1, beta2 < 1; lr, weight_decay finite;
 * 1.2e-38 <= eps <= 1e30.  The list is read before the call returns, and with
 * lr, step and seed is part of what a stream capture records: only c and the
 * tensors can change from replay to replay.  No workspace; the same call gives
 * the same bits. */
#define DION_STATE_F32   32
#define DION_STATE_8BIT  8
#define DION_ADAMW_BLOCK 64

typedef struct dion_adamw_tensor {
  float*      X;        /* n, updated in place */
  const void* G;        /* n, float32 or bfloat16 per g_dtype, read only */
  void*       M;        /* n float32 or n bytes, updated in place */
  void*       V;        /* n float32 or n bytes, updated in place */
  uint8_t*    S;        /* 2 ceil(n / DION_ADAMW_BLOCK) bytes, updated in place, or NULL */
  int64_t     n;
  double      weight_decay;
} dion_adamw_tensor;

int dion_adamw_step_batched(const dion_adamw_tensor* tensors, int count, double lr, double beta1,
                            double beta2, double eps, int64_t step, const float* grad_scale,
                            int state_bits, uint32_t seed, int g_dtype, void* stream);
int dion_adamw_step(float* X, const void* G, void* M, void* V, uint8_t* S, int64_t n, double lr,
                    double beta1, double beta2, double eps, double weight_decay, int64_t step,
                    const float* grad_scale, int state_bits, uint32_t seed, int g_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBDION_DION_H_ */
