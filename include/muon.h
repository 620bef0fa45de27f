/*
 * muon.h -- C ABI of the GB300 (sm_103a) Muon / Periodic Row-wise Muon optimizer step.
 *
 * What the library computes (per 2-D weight matrix W of shape A x B, row-major):
 *
 *   momentum      M <- mu*M + G
 *                 ("Muon is Scalable for LLM Training" notes, section 2.1, Eq. (1));
 *   Newton-Schulz X0 = M/||M||_F, five times X <- a X + b (X X^T) X + c (X X^T)^2 X,
 *                 (a, b, c) = (3.4445, -4.7750, 2.0315), run on the short side of M
 *                 (same page, section 2.1, Eq. (2); section 2.2 for N = 5);
 *   RowNorm       each of the min(A, B) lines of M along its long dimension scaled
 *                 to unit L2 norm: rows when A <= B, columns when A > B
 *                 ("Scaling Muon for Diffusion Transformers", abstract and the
 *                 Periodic Row-wise / distributed-implementation paragraphs);
 *   apply         W <- W - eta*(s*U + lambda*W) with s = 0.2*sqrt(max(A, B)) on NS5
 *                 steps and gamma*0.2*sqrt(max(A, B)) on RowNorm steps
 *                 ("Muon is Scalable" notes, Eq. (3), (4), (7));
 *   schedule      NS5 refresh iff step % K == 0 (step counted from 0), RowNorm
 *                 otherwise ("Scaling Muon for Diffusion Transformers", Periodic
 *                 Row-wise paragraph; K = 1 is vanilla Muon).
 *
 * Conventions for every entry point:
 *  - Memory: all tensor pointers are DEVICE pointers owned by the caller (for
 *    example PyTorch allocations).  The library allocates no device memory and
 *    frees nothing.  Scratch space comes from the caller's workspace `ws`
 *    (device, 256-byte aligned, at least muon_workspace_size() bytes).  A
 *    workspace holds one call's scratch: two calls whose GPU work may overlap
 *    (different streams, no ordering between them) need two workspaces.  Arrays
 *    of muon_matrix and arrays of output pointers are HOST arrays, read during
 *    the call only.
 *  - Layout: W, G, M, O and R are row-major A x B with leading dimension B (dense).
 *    M is always fp32.  W and G are fp32 or bf16 (MUON_DTYPE_*); within one call
 *    every matrix uses the same (w_dtype, g_dtype) pair.
 *  - Streams: `stream` is a cudaStream_t (NULL = legacy default stream).  Every
 *    call only enqueues work on it, never synchronises (except muon_check_status),
 *    and can be captured into a CUDA graph once the one-time set-up has run: the
 *    first call on a host thread and device creates a second stream and two
 *    events for that thread, and the first call on a device sets kernel attributes
 *    and queries occupancy.  Call muon_init() (or make one eager call) on each
 *    host thread and device before capturing the library's calls.
 *  - Errors: host-side validation happens before any launch; on error nothing is
 *    enqueued and a negative muon_status is returned.  Device-side failures
 *    (bounded waits that expired; non-finite norms when the finite check of
 *    muon_periodic_step_ex is on) are recorded in the workspace's status word and
 *    read by muon_check_status().
 *  - Non-finite values: NaN or Inf in G propagate through the arithmetic as IEEE
 *    defines it, deterministically.  A NaN or Inf in M makes ||M||_F (a refresh
 *    step) or that line's norm (a RowNorm step) non-finite; the direction is then
 *    M divided by that norm, so the whole matrix (refresh) or that line (RowNorm)
 *    of W becomes NaN, and an Inf norm turns the finite entries' direction into 0.
 *    Only an exactly zero norm is treated as a zero direction.
 *  - Matrices with A == 0 or B == 0 are accepted and skipped; n == 0 is a no-op.
 *  - Determinism: all reductions use a fixed order, so identical inputs give
 *    bit-identical outputs run to run.
 */
#ifndef MUON_GB300_MUON_H
#define MUON_GB300_MUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_ABI_VERSION 2

typedef enum muon_status {
  MUON_OK = 0,
  MUON_ERR_INVALID = -1,     /* bad argument: null pointer, negative size, K < 1, step < 0 */
  MUON_ERR_UNSUPPORTED = -2, /* dtype not supported, mixed dtypes, size beyond limits */
  MUON_ERR_WORKSPACE = -3,   /* workspace null, misaligned or smaller than required */
  MUON_ERR_CUDA = -4,        /* a CUDA runtime or driver call failed */
  MUON_ERR_TIMEOUT = -5,     /* a device-side bounded wait expired (from muon_check_status) */
  MUON_ERR_NO_DEVICE = -6,   /* no usable sm_103 device is current */
  MUON_ERR_NONFINITE = -7    /* a momentum norm was NaN or Inf (from muon_check_status, when the
                                finite check of muon_periodic_step_ex was on) */
} muon_status;

enum { MUON_DTYPE_F32 = 0, MUON_DTYPE_BF16 = 1 };

/* Newton-Schulz arithmetic: bf16 operands with fp32 accumulation on the tensor
 * cores (tcgen05), or fp32 throughout on the CUDA cores. */
enum { MUON_NS5_BF16 = 0, MUON_NS5_F32 = 1 };

/* Branch reported by muon_periodic_step. */
enum { MUON_BRANCH_ROWNORM = 0, MUON_BRANCH_NS5 = 1 };

typedef struct muon_matrix {
  void* W;          /* device, A x B row-major, w_dtype; updated in place           */
  const void* G;    /* device, A x B row-major, g_dtype; the step's gradient         */
  float* M;         /* device, A x B row-major, fp32 momentum; updated in place      */
  int64_t rows;     /* A (0 <= A < 2^31)                                             */
  int64_t cols;     /* B (0 <= B < 2^31)                                             */
  int32_t w_dtype;  /* MUON_DTYPE_F32 or MUON_DTYPE_BF16                             */
  int32_t g_dtype;  /* MUON_DTYPE_F32 or MUON_DTYPE_BF16                             */
} muon_matrix;

typedef void* muon_stream_t; /* cudaStream_t */

/* Bytes of workspace any entry point needs for this matrix list and NS5 mode
 * (the maximum over all entry points; one workspace serves them all).
 * Returns 0 for n == 0, and (size_t)-1 for an invalid list. */
size_t muon_workspace_size(const muon_matrix* mats, int n, int ns5_mode);

/* Momentum, Eq. (1) of the "Muon is Scalable" notes (section 2.1):
 *   M_i <- mu*M_i + G_i for every matrix.
 * fro_sq_out: optional device array of n floats; when non-NULL it receives
 * ||M_i||_F^2 of the updated momentum (fixed-order fp32 reduction), and ws must
 * be a valid workspace.  W is not read.  ws may be NULL when fro_sq_out is NULL. */
int muon_momentum(const muon_matrix* mats, int n, float mu, float* fro_sq_out,
                  void* ws, size_t ws_bytes, muon_stream_t stream);

/* Frobenius norm of the current momentum, the normaliser of X0 = M/||M||_F
 * (section 2.1 of the "Muon is Scalable" notes): fro_out[i] = ||M_i||_F (device,
 * n floats).  M is read only; G and W are not read. */
int muon_fro_norm(const muon_matrix* mats, int n, float* fro_out,
                  void* ws, size_t ws_bytes, muon_stream_t stream);

/* Same result as muon_fro_norm, for callers that cannot allocate device memory
 * (for example a plugin inside a host framework that owns every device
 * allocation, or code that must not call cudaMalloc mid-step because it would
 * synchronise the device).  The pages have no counterpart: this is a deployment
 * variant of the norm above.
 *  - No workspace: the per-tile partial sums live in a fixed 4 MiB array inside
 *    the library, resident on every GPU that loads it until the process exits.
 *  - Limit: at most 2^20 tiles of 64 x 128 elements per call (about 8.6e9
 *    elements of M in total); larger lists return MUON_ERR_UNSUPPORTED.
 *  - Every call looks up the array's device address on the current device
 *    (cudaGetSymbolAddress, which allocates nothing); the first call on a device
 *    may load the library's module there, so make that first call before any
 *    stream capture.  A device reset is handled: the next call finds the array
 *    again.
 *  - Same argument checks and status codes as muon_fro_norm (dtypes included).
 *  - All calls share the array.  Calls that overlap on the GPU (different
 *    streams, or different host threads) race on it; serialise them.
 *  - Allocates nothing, reads M only, writes fro_out[i] = ||M_i||_F.  Does not
 *    update muon_launch_count. */
int muon_fro_norm_noalloc(const muon_matrix* mats, int n, float* fro_out, muon_stream_t stream);

/* Newton-Schulz-5 of the current momentum, Eq. (2) of the "Muon is Scalable"
 * notes: O_i = NS5(M_i), computed on the short side of M_i and returned in
 * M_i's A x B orientation.  O_out: host array of n device pointers, each an
 * A x B row-major buffer of o_dtype.  ns5_mode selects the arithmetic
 * (MUON_NS5_BF16: bf16 tensor-core GEMMs, fp32 accumulate, bf16 intermediates;
 * MUON_NS5_F32: fp32 throughout).  M, G and W are not modified.  A zero M gives
 * O = 0. */
int muon_ns5_batched(const muon_matrix* mats, int n, int ns5_mode, void* const* O_out,
                     int o_dtype, void* ws, size_t ws_bytes, muon_stream_t stream);

/* RowNorm of the current momentum (Periodic Row-wise branch): R_i = M_i with each
 * row (A <= B) or each column (A > B) scaled to unit L2 norm; a zero line stays
 * zero.  R_out: host array of n device pointers to fp32 A x B buffers.  M is
 * read only. */
int muon_rownorm(const muon_matrix* mats, int n, float* const* R_out,
                 void* ws, size_t ws_bytes, muon_stream_t stream);

/* Apply, Eq. (4)/(7) of the "Muon is Scalable" notes:
 *   W_i <- W_i - eta*(scale_mul*sqrt(max(A, B))*U_i + lambda*W_i)
 * computed in fp32 with one rounding to w_dtype.  U: host array of n device
 * pointers to A x B buffers of u_dtype.  scale_mul is 0.2 for an NS5 direction
 * and 0.2*gamma for a RowNorm direction. */
int muon_apply(const muon_matrix* mats, int n, const void* const* U, int u_dtype,
               float scale_mul, float eta, float lambda, muon_stream_t stream);

/* One Periodic Row-wise Muon step over every matrix (K = 1: vanilla Muon):
 *   refresh = (step % K == 0);
 *   M <- mu*M + G;
 *   U = NS5(M) (refresh) or RowNorm(M) (otherwise);
 *   W <- W - eta*(s*U + lambda*W), s = 0.2*sqrt(max(A, B)), times gamma when not refreshing.
 * On refresh steps the apply is fused into the last Newton-Schulz GEMM.  On
 * RowNorm steps, wide and square matrices take one pass over memory (momentum,
 * row norms and apply); tall matrices take two row-contiguous passes in one
 * launch, the second re-reading the new momentum from L2.  The wide-row kernels
 * of a RowNorm step run on a second stream owned by the library (one per host
 * thread and device), forked from and joined back to `stream` with events, so
 * the call stays ordered on `stream` and capturable.  branch_out (host,
 * optional) receives MUON_BRANCH_NS5 or MUON_BRANCH_ROWNORM. */
int muon_periodic_step(const muon_matrix* mats, int n, int64_t step, int K, float gamma,
                       float mu, float eta, float lambda, int ns5_mode, void* ws,
                       size_t ws_bytes, muon_stream_t stream, int* branch_out);

/* One-time set-up for the current device and the calling host thread: checks the
 * device (sm_103), creates the thread's second stream and its fork/join events, sets
 * the tensor-core kernels' shared-memory attributes and caches occupancy figures.
 * Every entry point does the same on its first use; calling muon_init first makes
 * the first step capturable into a CUDA graph.  Allocates no device memory;
 * repeated calls are cheap no-ops.  Returns MUON_ERR_NO_DEVICE without a usable
 * device, MUON_ERR_CUDA if a set-up call fails. */
int muon_init(void);

/* Clears the status header of a fresh workspace (the first 256 bytes) on
 * `stream`.  Call once after allocating a workspace whose contents are not
 * already zero; the rest of the workspace needs no initialisation. */
int muon_workspace_init(void* ws, size_t ws_bytes, muon_stream_t stream);

/* Update scale of muon_periodic_step_ex. */
enum {
  MUON_SCALE_ADJUSTED_LR = 0, /* s = 0.2*sqrt(max(A, B)) ("Muon is Scalable" notes, Eq. (4)/(7)) */
  MUON_SCALE_UPDATE_NORM = 1  /* s = 0.2/RMS(U), "Update Norm", same notes, section 3.1, Eq. (6);
                                 on RowNorm steps the RMS is over the lines that carry the update,
                                 so it equals the Eq. (7) scale unless a line of M is zero */
};

typedef struct muon_step_options {
  int scale_mode;      /* MUON_SCALE_* */
  float* update_rms;   /* optional device array of n floats: RMS of each matrix's direction U
                          (the Newton-Schulz output, or the RowNorm of M) over its A*B elements,
                          as monitored against Lemma 1 ("Muon is Scalable" notes, section 2.2) */
  int check_finite;    /* nonzero: the kernels that reduce the momentum's norms (||M||_F^2 on a
                          refresh step, every line's sum of squares on a RowNorm step) set a bit
                          in the workspace status word when one is NaN or Inf, which
                          muon_check_status returns as MUON_ERR_NONFINITE.  The check reads
                          values the step computes anyway: it adds no memory traffic.  The
                          step's results are the same with the check on or off. */
} muon_step_options;

/* muon_periodic_step with options (opts == NULL: Eq. (4)/(7) scale, no telemetry).
 * With MUON_SCALE_UPDATE_NORM, refresh steps write O to the workspace, reduce its
 * sum of squares in a fixed order, then apply W <- W - eta*(0.2*O/RMS(O) + lambda*W)
 * in a separate pass (a zero O gives pure weight decay). */
int muon_periodic_step_ex(const muon_matrix* mats, int n, int64_t step, int K, float gamma,
                          float mu, float eta, float lambda, int ns5_mode,
                          const muon_step_options* opts, void* ws, size_t ws_bytes,
                          muon_stream_t stream, int* branch_out);

/* A parameter that Muon does not update (bias, normalisation weight, out-of-block
 * parameter), with its AdamW state. */
typedef struct muon_adamw_param {
  void* P;          /* device, numel elements of p_dtype; updated in place            */
  const void* G;    /* device, numel elements of g_dtype                             */
  float* m;         /* device, numel fp32 first moment (starts at 0)                 */
  float* v;         /* device, numel fp32 second moment (starts at 0)                */
  int64_t numel;
  int32_t p_dtype;  /* MUON_DTYPE_F32 or MUON_DTYPE_BF16                             */
  int32_t g_dtype;  /* MUON_DTYPE_F32 or MUON_DTYPE_BF16                             */
} muon_adamw_param;

/* AdamW on the parameters beside the Muon matrices ("Scaling Muon for Diffusion
 * Transformers", summary page: bias, normalisation and out-of-block parameters
 * keep AdamW, an auxiliary group at LR 1e-4; "Muon is Scalable" notes, section
 * 2.2: the two optimizers share learning rate and weight decay):
 *   m <- b1*m + (1-b1)*g;  v <- b2*v + (1-b2)*g^2;
 *   p <- p - lr*( (m/(1-b1^t)) / (sqrt(v/(1-b2^t)) + eps) + weight_decay*p ),
 * fp32 arithmetic, one rounding to p_dtype (beta1 and beta2 are double so that 1-beta
 * is exact enough: 0.999 in fp32 would put 1.3e-5 into 1-beta2).  t counts steps from 1.  One launch
 * covers the whole list (host array); every entry uses the same dtype pair. */
int muon_adamw_step(const muon_adamw_param* params, int n, int64_t t, float lr, double beta1,
                    double beta2, float eps, float weight_decay, muon_stream_t stream);

/* ---------------------------------------------------------------------------
 * The operators at a model's head: the parameters that Muon leaves to AdamW are
 * mostly the norms and the vocabulary matrix.  These entry points compute the last
 * part of a training step around them -- layer norm, the vocabulary projection with
 * its loss, and an AdamW step with 8-bit moments.  The conventions above hold for
 * them too; the pages have no counterpart for them.
 * Strides (ld*) are in elements between rows; columns are contiguous. */

/* Layer norm over the last dimension, for rows r = 0 .. rows-1:
 *   mean = sum(x)/dim;  rstd = 1/sqrt(sum((x - mean)^2)/dim + eps);
 *   y = (x - mean)*rstd*weight + bias.
 * x and y are x_dtype, weight and bias w_dtype (either may be NULL: 1 and 0).  mean
 * and rstd are fp32, one a row, and may be NULL when no backward pass follows.
 * Arithmetic is fp32 with one rounding of y; the variance is summed from the centred
 * values.  y may be x itself (same ld); other overlaps are not allowed.
 * eps >= 0; rows and dim at most 2^30, dim >= 1; rows == 0 is a no-op. */
int muon_layernorm_forward(const void* x, int64_t ldx, const void* weight, const void* bias,
                           int64_t rows, int64_t dim, int x_dtype, int w_dtype, float eps,
                           void* y, int64_t ldy, float* mean, float* rstd, muon_stream_t stream);

/* Bytes of workspace muon_layernorm_backward needs to reduce the weight's and bias's
 * gradients; (size_t)-1 for invalid sizes. */
size_t muon_layernorm_workspace_size(int64_t rows, int64_t dim);

/* Gradient of the above.  With xh = (x - mean)*rstd and g = dy*weight:
 *   dx = rstd*(g - sum(g)/dim - xh*sum(g*xh)/dim);
 *   dweight = sum over rows of dy*xh;  dbias = sum over rows of dy.
 * mean and rstd are the forward pass's.  dy and dx are x_dtype; dweight and dbias are
 * w_dtype, overwritten, and may each be NULL; rows == 0 writes zeros to them.  The
 * sums over rows are fp32 in a fixed order.  dx may be dy itself (same ld).  ws may
 * be NULL when dweight and dbias both are. */
int muon_layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight,
                            const float* mean, const float* rstd, int64_t rows, int64_t dim,
                            int x_dtype, int w_dtype, void* dx, int64_t lddx, void* dweight, void* dbias,
                            void* ws, size_t ws_bytes, muon_stream_t stream);

/* Softmax cross entropy of the logits z = H W^T over a vocabulary, computed in pieces
 * so that the rows x vocab logits are never kept. */
typedef struct muon_linear_ce {
  const void* H;          /* device, rows x dim, dtype; the hidden states                      */
  const void* W;          /* device, vocab x dim, dtype; the vocabulary matrix                 */
  const int64_t* labels;  /* device, rows                                                      */
  int64_t rows, vocab, dim; /* rows >= 0, vocab >= 1, dim >= 1, each at most 2^30              */
  int64_t ldh, ldw;       /* elements between rows of H and of W (>= dim)                      */
  int32_t dtype;          /* of H, W and their gradients: MUON_DTYPE_F32 or MUON_DTYPE_BF16    */
  int64_t ignore_index;   /* rows with this label carry no loss and no gradient                */
} muon_linear_ce;

/* Bytes of workspace for muon_linear_ce_forward (backward == 0) or for both passes
 * (backward != 0) of these sizes, strides, dtype and pointers (NULL pointers count as
 * aligned).  It holds room for a copy of H, for one of W where W's rows do not start on
 * 16-byte boundaries (both three bf16 parts long for 32-bit operands), and for the
 * backward pass two pieces of g (at most 512 MB each, but 2048 columns of the vocabulary
 * at least) and fp32 sums of dH.  (size_t)-1 for invalid sizes. */
size_t muon_linear_ce_workspace_size(const muon_linear_ce* a, int backward);

/* loss[r] = lse[r] - z[r, label_r] with lse[r] = log(sum_v exp(z[r, v])); loss is 0 for
 * an ignored row, whose lse is computed all the same.  A label outside [0, vocab) that
 * is not ignore_index makes that row's loss NaN.  stats, if not NULL: stats[0] the mean
 * loss over the rows that are not ignored (0 if there is none), stats[1] their count.
 * loss, lse and stats are device fp32.  Products of bf16 values are exact and summed in
 * fp32; a NaN or +Inf logit makes the row's lse and loss NaN.  Call muon_workspace_init
 * once on a fresh workspace; muon_check_status reports an expired wait.  Until it has done
 * so, this call and the next ones with the workspace write NaN to every output (the
 * backward pass too), so that a caller who does not ask cannot take them for results. */
int muon_linear_ce_forward(const muon_linear_ce* a, float* loss, float* lse, float* stats,
                           void* ws, size_t ws_bytes, muon_stream_t stream);

/* Gradient of u * sum_r c_r*loss[r]:  g[r, v] = c_r*(exp(z[r, v] - lse[r]) - [v == label_r]),
 *   dH = u g W  (rows x dim, leading dimension dim),  dW = u g^T H  (vocab x dim, likewise),
 * both of a->dtype and overwritten; either may be NULL.  c_r = row_grad ? row_grad[r] : 1,
 * and 0 for an ignored row and for one whose label is out of range, whatever such a row
 * of H, lse and row_grad holds (NaN and infinities included).
 * u = grad_scale * (upstream ? upstream[0] : 1) * (stats ? 1/max(stats[1], 1) : 1): with the
 * forward pass's stats this is the gradient of grad_scale * upstream * the mean loss.
 * row_grad, upstream and stats are device fp32.  The logits are computed again, by pieces
 * of the vocabulary.  In bf16, g is rounded to bf16 before the two products, which are
 * summed in fp32 and scaled by u before their rounding (a factor that every row shares is
 * better there: inside g its rounding would be the same for all of them). */
int muon_linear_ce_backward(const muon_linear_ce* a, const float* lse, const float* row_grad,
                            const float* stats, const float* upstream, float grad_scale, void* dH,
                            void* dW, void* ws, size_t ws_bytes, muon_stream_t stream);

/* Log probabilities of given tokens, entropies and the likeliest alternatives under the
 * softmax of the logits z = H W^T, which are never kept.  Scoring, decoding and
 * policy-gradient training take these; a->labels holds the tokens (NULL, forward only: no
 * token is given, every row counts).
 *   lse[r] = log(sum_v exp(z[r, v]));  logprob[r] = z[r, token_r] - lse[r];
 *   entropy[r] = -sum_v p log p,  p = exp(z[r, v] - lse[r]);
 *   ids[r][0 .. top): the `top` largest logits, equal ones by the lower id;
 *   alternatives[r][0 .. top): their log probabilities.
 * A row with token ignore_index has logprob and entropy 0, ids -1 and alternatives minus
 * infinity (lse is computed); a token outside [0, vocab) that is not ignore_index makes
 * logprob and entropy NaN.  Logits of minus infinity, or below -2^120 (a mask of the type's
 * lowest value), are masked entries: they are no alternatives, and places without one hold
 * -1 and minus infinity.  A row of nothing but minus infinities has lse minus infinity,
 * logprob and entropy NaN and no alternatives; a NaN or +Inf logit makes the row's lse,
 * logprob, entropy and alternatives NaN and its ids -1.  Logits are summed as for the cross
 * entropy.  Those that can be among the largest, by a bound on their error (a share of the
 * lengths of their rows of H and W, so that terms that cancel are allowed for), are summed again, to 2^-45 of their
 * largest partial sum, and ranked by that.  logprob, entropy, lse
 * and alternatives are device fp32, ids device int64.  logprob may be NULL without tokens,
 * ids and alternatives with top == 0. */
#define MUON_LOGPROB_MAX_TOP 32
int muon_linear_logprob_forward(const muon_linear_ce* a, int top, float* logprob, float* entropy, float* lse,
                                int64_t* ids, float* alternatives, void* ws, size_t ws_bytes,
                                muon_stream_t stream);

/* Bytes of workspace for muon_linear_logprob_forward with so many alternatives (backward ==
 * 0) or for both passes; (size_t)-1 for invalid arguments.  The rules of
 * muon_linear_ce_workspace_size hold (initialisation, status and expired waits, too). */
size_t muon_linear_logprob_workspace_size(const muon_linear_ce* a, int top, int backward);

/* Gradient of sum_r (g_logprob[r]*logprob[r] + g_entropy[r]*entropy[r]):
 *   g[r, v] = g_logprob[r]*([v == token_r] - p) - g_entropy[r]*p*(log p + entropy[r]),
 *   dH = g W,  dW = g^T H, as for the cross entropy (in bf16, g is rounded to bf16).
 * g_logprob or g_entropy may be NULL (zeros; entropy may be NULL with g_entropy).  lse and
 * entropy are the forward pass's.  A row with token ignore_index, or with one out of range,
 * has no gradient, whatever it holds.  Alternatives have no gradient. */
int muon_linear_logprob_backward(const muon_linear_ce* a, const float* lse, const float* entropy,
                                 const float* g_logprob, const float* g_entropy, void* dH, void* dW, void* ws,
                                 size_t ws_bytes, muon_stream_t stream);

/* Root-mean-square norm over the last dimension, behind a residual's addition:
 *   t = x + residual, rounded to x_dtype (t = x without a residual);
 *   rstd = 1/sqrt(sum(t^2)/dim + eps);  y = t*rstd*weight.
 * x, residual, total (t) and y are x_dtype, weight (NULL: 1) is w_dtype.  total may be NULL,
 * and is without a residual; it may be x or residual itself (same ld), y may be x itself
 * where total is not; other overlaps are not allowed.  rstd (fp32, one a row) may be NULL.
 * With codes, y is also written in 8 bits (y itself may then be NULL): for each row and
 * MUON_RMS_GROUP columns (the last group may be shorter) a scale
 *   s = max(max|y|/448, 2^-100)   (fp32, rounded to nearest; rows x ceil(dim/128), contiguous)
 * and e4m3 codes of the fp32 quotient y/s, rounded to nearest, ties to even: code*s stands for y.  A NaN
 * among a group's y makes its scale and codes NaN.  Arithmetic is fp32, with one rounding
 * of y.  eps >= 0; rows and dim at most 2^30, dim >= 1; rows == 0 is a no-op. */
#define MUON_RMS_GROUP 128
int muon_rmsnorm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                         int64_t rows, int64_t dim, int x_dtype, int w_dtype, float eps, void* total, int64_t ldt,
                         void* y, int64_t ldy, uint8_t* codes, int64_t ldc, float* scales, float* rstd,
                         muon_stream_t stream);

/* Bytes of workspace muon_rmsnorm_backward needs to reduce the weight's gradient;
 * (size_t)-1 for invalid sizes. */
size_t muon_rmsnorm_workspace_size(int64_t rows, int64_t dim);

/* Gradient of y (and of total) with respect to t, which x and residual share.  With xh =
 * t*rstd and g = dy*weight:
 *   dx = dtotal + rstd*(g - xh*sum(g*xh)/dim);  dweight = sum over rows of dy*xh.
 * total is the forward pass's t (x itself without a residual), dtotal the gradient that
 * total has from elsewhere (NULL: 0).  dy, dtotal and dx are x_dtype; dweight is w_dtype,
 * overwritten, and may be NULL (ws too then); rows == 0 writes zeros to it.  The sums over
 * rows are fp32 in a fixed order.  dx may be dy or dtotal itself (same ld). */
int muon_rmsnorm_backward(const void* dy, int64_t lddy, const void* total, int64_t ldt, const void* weight,
                          const float* rstd, const void* dtotal, int64_t lddt, int64_t rows, int64_t dim,
                          int x_dtype, int w_dtype, void* dx, int64_t lddx, void* dweight, void* ws,
                          size_t ws_bytes, muon_stream_t stream);

/* A gradient of the list that muon_clip_grad_norm takes. */
typedef struct muon_grad {
  void* G;           /* device, numel contiguous elements, scaled in place            */
  int64_t numel;     /* >= 0, below 2^42                                              */
  int32_t dtype;     /* MUON_DTYPE_F32 or MUON_DTYPE_BF16                             */
  int32_t reserved;
} muon_grad;

/* The global norm of n gradients (host array; of both dtypes), and clipping by it:
 *   norm = sqrt(sum of the squares of all elements);
 *   where norm > max_norm:  g <- g*(max_norm/norm), rounded to g's dtype.
 * norm is one device fp32 number, of the gradients as they were.  max_norm >= 0; an infinite
 * one computes the norm alone.  Squares are added in fp32 by 64 and in 64 bits above that,
 * with a power of two taken out where fp32 would overflow or underflow, in a fixed order.
 * As the formula says, a norm of infinity makes finite gradients 0 and infinite ones NaN, and
 * a NaN norm makes all of them NaN.  Tensors that are scaled must not share memory
 * (MUON_ERR_INVALID).  ws: muon_clip_workspace_size() bytes, 8-byte aligned, no
 * initialisation; one call at a time uses it. */
size_t muon_clip_workspace_size(void);
int muon_clip_grad_norm(const muon_grad* grads, int n, double max_norm, float* norm, void* ws, size_t ws_bytes,
                        muon_stream_t stream);

/* AdamW with both moments held in 8 bits.  Blocks of MUON_ADAMW8_BLOCK consecutive
 * elements share one scale byte s per moment.  A code c stands for the fp32 number
 * whose bits are (c + base) << 20, so for a float with 3 bits of mantissa:
 *   first moment   1 sign bit and 7 bits c, base = 8*max(s - 16, 0): 15.9 binades a block;
 *   second moment  8 bits c,                base = 8*max(s - 32, 0): 31.9 binades a block;
 * c = 0 stands for 0, whatever s; the first moment's byte 0x80 stands for NaN.  s is the
 * smallest that holds the block's largest value.  New moments are rounded
 * stochastically, up with a probability equal to the remainder (16 bits), because one
 * step moves the second moment by 1 - beta2, far less than the grid's spacing, and
 * rounding to nearest would hold it still.  A nonzero second moment never rounds to 0
 * (it would turn the update into m/eps): it takes code 1 at least.  The random bits
 * depend only on (seed, t, index of the element), so a step is reproducible bit for bit.
 * A fresh state is all zero bytes. */
#define MUON_ADAMW8_BLOCK 128
typedef struct muon_adamw8_param {
  void* P;           /* device, numel elements of p_dtype; updated in place                    */
  const void* G;     /* device, numel elements of g_dtype                                      */
  uint8_t* m;        /* device, 16-byte aligned, ceil(numel/128)*128 codes of the first moment */
  uint8_t* v;        /* the same for the second moment                                         */
  uint8_t* m_scale;  /* device, ceil(numel/128) scale bytes                                    */
  uint8_t* v_scale;
  int64_t numel;
  int64_t first;     /* index of the first element for the random bits: a multiple of 128; give
                        every parameter a range of its own                                     */
  int32_t p_dtype;   /* MUON_DTYPE_F32 or MUON_DTYPE_BF16                                      */
  int32_t g_dtype;   /* MUON_DTYPE_F32 or MUON_DTYPE_BF16                                      */
} muon_adamw8_param;

/* The update of muon_adamw_step, from the new moments before they are rounded to 8 bits,
 * fp32 arithmetic and one rounding to p_dtype.  Codes past numel in the last block are
 * set to 0.  A NaN or Inf gradient makes that element's m and P NaN and leaves its
 * block's other elements as they would be; a second moment beyond fp32 is held at its
 * largest code.  One launch per 256 parameters; every entry uses the same dtype pair. */
int muon_adamw8_step(const muon_adamw8_param* params, int n, int64_t t, float lr, double beta1,
                     double beta2, float eps, float weight_decay, uint32_t seed, muon_stream_t stream);

/* The values that codes stand for, as bf16 (exact): numel codes, a multiple of
 * MUON_ADAMW8_BLOCK.  m and v 16-byte aligned, m_out and v_out 32-byte aligned; m with
 * m_scale and m_out, or v with v_scale and v_out, may be NULL. */
int muon_adamw8_unpack(const uint8_t* m, const uint8_t* m_scale, const uint8_t* v, const uint8_t* v_scale,
                       int64_t numel, void* m_out, void* v_out, muon_stream_t stream);

/* Synchronises `stream`, reads and clears the device status word in `ws`, and
 * returns MUON_OK or the recorded error: MUON_ERR_TIMEOUT when a bounded wait
 * expired (it takes precedence), else MUON_ERR_NONFINITE when the finite check saw
 * a NaN or Inf norm.  The word accumulates over calls until it is read. */
int muon_check_status(void* ws, size_t ws_bytes, muon_stream_t stream);

/* Profiling hook (process-wide): up to 5 cudaEvent_t handles that
 * muon_periodic_step records on its stream at phase boundaries:
 *   [0] refresh step start, [1] first Newton-Schulz GEMM launch,
 *   [2] after the last Newton-Schulz GEMM, [3] RowNorm step start,
 *   [4] RowNorm step end.
 * NULL entries are skipped; n == 0 turns the hook off.  Recording also works
 * under stream capture (the records become graph nodes). */
int muon_profile_events(void* const* events, int n);

/* Number of kernels that the most recent entry-point call made by this host
 * thread enqueued (0 after a validation error). */
int muon_launch_count(void);

/* Static description of a status code. */
const char* muon_status_str(int status);

/* MUON_ABI_VERSION of the loaded library. */
int muon_abi_version(void);

/* Test hooks (process-wide, not for production use).
 * timeout_ms: limit of every device-side wait (default 4000 ms; 0 restores it).
 * flags: MUON_DEBUG_STALL_PRODUCER makes the tensor-core GEMM's load warp issue
 * nothing, and the tall-matrix RowNorm kernel publish no column norms, so that
 * their consumers' bounded waits expire and report MUON_ERR_TIMEOUT through
 * muon_check_status (no fault, no hang).
 * Tall matrices of RowNorm steps normally take two row-contiguous passes whose
 * second pass re-reads the new momentum from L2.  MUON_DEBUG_NO_CLUSTER sends
 * them through the plain two-pass kernels instead, MUON_DEBUG_TALL_CLUSTER
 * through the single-pass thread-block-cluster kernel (to test every path).
 * MUON_DEBUG_NO_OVERLAP runs the wide-row and tall-column kernels of a RowNorm
 * step one after the other on the caller's stream instead of side by side.
 * MUON_DEBUG_NO_PAIR runs the tensor-core Newton-Schulz GEMMs with one CTA per
 * 128 x 256 tile instead of 2-CTA clusters (tcgen05 cta_group::2) on 256 x 256 tiles.
 * MUON_DEBUG_CE_PIECE times n (1 .. 255) cuts the vocabulary of the linear cross entropy's
 * backward pass into pieces of 256 n columns, in the workspace's size and in the call, so
 * that small cases have several. */
enum {
  MUON_DEBUG_STALL_PRODUCER = 1,
  MUON_DEBUG_NO_CLUSTER = 2,
  MUON_DEBUG_NO_OVERLAP = 4,
  MUON_DEBUG_TALL_CLUSTER = 8,
  MUON_DEBUG_NO_PAIR = 16,
  MUON_DEBUG_CE_PIECE = 256
};
int muon_debug_set(int flags, int timeout_ms);

#ifdef __cplusplus
}
#endif
#endif /* MUON_GB300_MUON_H */
