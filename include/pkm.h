/*
 * pkm.h -- C ABI of the product-key memory (PKM) layer library for NVIDIA B200
 * (sm_100a). Library file: libpkm.so (product_key_memory_b200/libpkm.so).
 *
 * The layer is the one of "Large Memory Layers with Product Keys" (Lample et al.,
 * 2019). Per token and head (gptget.net summary of that paper, Methodology and the
 * Deep Analysis / Methodology list; "Product Keys Give Transformers Million-Slot
 * Memory Layers", sections "Why top-k of each half is enough" and "Implied keys
 * vs stored sub-keys"):
 *   q      = BN(x W_q^T)                query network: linear map + inference BatchNorm
 *   q1, q2 = the two halves of q_h      (dq/2 each)
 *   s1, s2 = q1 C_h^T, q2 C'_h^T        score every sub-key of each codebook
 *   keep the top-k of s1 and of s2
 *   score(i, j) = s1[i] + s2[j] over the k x k pairs; keep the exact top-k keys;
 *   the key (i, j) has flat slot i*n + j
 *   w      = softmax over the k kept scores
 *   out[t] = sum over heads h, kept j of w[t,h,j] * V[slot[t,h,j]]
 * Orders: every top-k is by score descending, ties to the lower id (sub-key id in
 * the per-half lists, flat slot in the final list). Output lists are sorted in that
 * order.
 *
 * Conventions for every entry point:
 *   - Tensors are caller-owned DEVICE pointers, row-major and contiguous, 16-byte
 *     aligned. The library allocates no device memory: scratch is the caller's
 *     `workspace` (pkm_backward_values_noalloc alone uses a fixed array compiled
 *     into the library).
 *   - Persistent state the library keeps: two process-wide option values
 *     (pkm_set_option), the tensor-map encoder's address and the SM count (looked
 *     up once), each kernel's raised shared-memory limit, and, only while tracing
 *     is on, a pool of timing events. A forward pipelined over sub-batches
 *     (PKM_OPT_SUBBATCHES > 1) also creates, on first use per device, one helper
 *     stream and a pool of ordering events; the default forward (one batch) uses
 *     neither and issues its three kernels on `stream` alone.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     All work is enqueued asynchronously and ordered on it; no call synchronises.
 *   - Arguments are validated before anything is launched: a call that returns an
 *     error has launched nothing and written nothing.
 *   - Kernels that wait on hardware barriers give up after a bounded time (1 s)
 *     and record it in the workspace's status word, as do gathers that meet a slot
 *     id outside [0, n*n) (skipped); pkm_device_status() waits for the stream and
 *     returns PKM_ERR_DEVICE if either happened.
 */
#ifndef PKM_H_
#define PKM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of x, W_q, sub-keys, values and grad_out. BN vectors, scores,
 * weights, out and gradients are always fp32. */
typedef enum { PKM_F32 = 0, PKM_BF16 = 1 } pkm_dtype;

/* Status codes. */
enum {
  PKM_OK = 0,
  PKM_ERR_INVALID_ARG = -1, /* NULL pointer, size out of range, k > n, odd dq, n*n > 2^31-1 */
  PKM_ERR_UNSUPPORTED = -2, /* valid layer this library does not run (k > 32, v not a multiple of
                               16 bytes, misaligned pointer) */
  PKM_ERR_WORKSPACE = -3,   /* workspace NULL or smaller than pkm_workspace_size() */
  PKM_ERR_CUDA = -4,        /* a CUDA runtime call or kernel launch failed */
  PKM_ERR_DEVICE = -5       /* a kernel recorded a device-side error: a bounded wait ran
                               out, or a slot id outside [0, n*n) was read */
};

/* Layer sizes. */
typedef struct {
  int64_t B;       /* tokens (rows of x); 0 is allowed, launches nothing, and then the
                      per-token pointers (x, out, indices, weights, scores, grad_out,
                      grad_scores) may be NULL */
  int32_t d_model; /* input width of the query network */
  int32_t H;       /* heads */
  int32_t dq;      /* query size per head, even; each half is dq/2 */
  int32_t n;       /* sub-keys per codebook; the memory has n*n slots */
  int32_t k;       /* keys kept per half and per head, 1 <= k <= min(n, 32) */
  int32_t v;       /* value width */
  int32_t dtype;   /* pkm_dtype of x, W_q, sub-keys, values, grad_out */
  float bn_eps;    /* BatchNorm epsilon (PyTorch's default is 1e-5) */
} pkm_shape;

/*
 * Bytes of workspace pkm_forward (for_backward = 0), pkm_backward_values
 * (for_backward = 1), pkm_slot_usage (for_backward = 2), pkm_backward or
 * pkm_backward_train (for_backward = 3) or pkm_forward_train (for_backward = 4) needs
 * for this shape; 0 if the shape is invalid.
 */
size_t pkm_workspace_size(const pkm_shape* s, int for_backward);

/*
 * Forward pass of the PKM layer (the steps listed at the top of this file).
 *
 *   x        [B][d_model]            dtype
 *   W_q      [H*dq][d_model]         dtype   (q = x W_q^T; no bias)
 *   bn_mean, bn_var, bn_gamma, bn_beta  [H*dq] fp32 running statistics and affine
 *            q = (acc - mean) / sqrt(var + bn_eps) * gamma + beta
 *   subkeys  [H][2][n][dq/2]         dtype   ([h][0] = C scores q1, [h][1] = C' scores q2)
 *   values   [n*n][v]                dtype   (one table shared by all heads)
 * Outputs (overwritten):
 *   out      [B][v]     fp32   sum over heads of the weighted value rows
 *   indices  [B][H][k]  int32  flat slots i*n + j, best first
 *   weights  [B][H][k]  fp32   softmax of the kept scores
 *   scores   [B][H][k]  fp32   kept key scores s1[i] + s2[j]; may be NULL
 * workspace: device scratch of at least pkm_workspace_size(s, 0) bytes, 256-byte
 *   aligned; its contents on entry do not matter.
 * Small batches take the small-batch path, which spreads W_q, the sub-keys and the
 * heads over all SMs for latency: up to 384 tokens with H <= 4 and 240 with H <= 8 on
 * bf16 layers with d_model and dq/2 multiples of 32 and dq/2 <= 256 (whose query
 * network and per-half scores there run as warp-level tensor-core tiles of 16 tokens),
 * up to 112 / 96 tokens otherwise; a pinned form (PKM_OPT_PATH small_fused /
 * small_split) takes up to 512 tokens for any H <= 8. By default it is three kernels
 * that overlap through programmatic dependent launch on `stream`: the first waits on
 * the device for the stream's earlier work and clears the status word itself, so
 * back-to-back calls overlap too. PKM_PATH_SMALL_FUSED runs it as one cooperative
 * kernel instead (one block per SM, its query, scoring and gather phases separated by
 * grid-wide barriers whose waits are bounded like the pipelines'). Up to 4 tokens
 * with H <= 4 (8 tokens on layers without the tensor-core tiles) the query and
 * scoring stages give a warp one W_q row or 8 sub-keys for all tokens, its lanes
 * splitting the dot products (rows of 16-byte multiples). Larger batches run
 * three kernels on `stream` (query network, per-half scores and top-k, candidate
 * top-k + softmax + gather). With PKM_OPT_SUBBATCHES > 1, large batches of
 * tensor-core shapes are processed in up to that many sub-batches; the value gather
 * of one sub-batch then runs on the library's helper stream (one per device) while
 * the next sub-batch is scored on `stream`. Event waits order both
 * ways, so all of the call's work is complete when `stream` reaches the point after
 * the call.
 * Returns PKM_OK or a status code above.
 */
int pkm_forward(const pkm_shape* s, const void* x, const void* W_q, const float* bn_mean,
                const float* bn_var, const float* bn_gamma, const float* bn_beta,
                const void* subkeys, const void* values, float* out, int32_t* indices,
                float* weights, float* scores, void* workspace, size_t workspace_bytes,
                void* stream);

/*
 * Sparse value backward ("trained end-to-end with sparse updates"; only the kept
 * slots receive gradient). With L = <grad_out, out>:
 *   grad_scores[t,h,j] = w_j * (g_j - sum_l w_l g_l),  g_j = <grad_out[t], V[slot_j]>
 *   grad_values[slot] += sum over picks (t,h,j) of that slot of w[t,h,j] * grad_out[t]
 *
 *   values      [n*n][v]   dtype
 *   indices     [B][H][k]  int32  (as written by pkm_forward; each in [0, n*n))
 *   weights     [B][H][k]  fp32
 *   grad_out    [B][v]     dtype
 *   grad_values [n*n][v]   fp32   ACCUMULATED into (the caller zeroes it once)
 *   grad_scores [B][H][k]  fp32   overwritten; may be NULL
 * Picks are grouped by slot with a stable radix sort, so each slot's picks are summed
 * in pick order and each touched row is read and written once, whatever the number of
 * picks that hit it (large groups are split over several blocks whose partial sums are
 * added in a fixed order). The result is bit-for-bit the same on every run, and no
 * row is updated with atomics. Slot ids outside [0, n*n) are skipped and counted in
 * the status word (PKM_ERR_DEVICE).
 * Only B, H, n, k, v and dtype of the shape are read; d_model, dq and bn_eps are
 * ignored.
 * With grad_scores requested, the sort of the picks by slot runs on the library's
 * helper stream (one per device, highest priority) while grad_scores is computed on
 * `stream`, and the row sums follow on `stream`; event waits order both ways, so all
 * of the call's work is complete when `stream` reaches the point after the call
 * (CUDA-graph capture of `stream` takes the helper stream's work in with it).
 * workspace: at least pkm_workspace_size(s, 1) bytes, 256-byte aligned.
 */
int pkm_backward_values(const pkm_shape* s, const void* values, const int32_t* indices,
                        const float* weights, const void* grad_out, float* grad_values,
                        float* grad_scores, void* workspace, size_t workspace_bytes,
                        void* stream);

/*
 * Full backward of the layer ("Large Memory Layers with Product Keys", Methodology:
 * the memory is trained end-to-end with the rest of the network). The top-k choice
 * is piecewise constant, so the picks of the forward are held fixed. With
 * L = <grad_out, out>, g_c the kept-score gradients of pkm_backward_values, key
 * (i, i') = slot i*n + i', acc = x W_q^T and s = gamma / sqrt(var + eps):
 *   dL/dq1_h = sum_j g_c[j] C_h[i_j],  dL/dq2_h = sum_j g_c[j] C'_h[i'_j]
 *   grad_subkeys[h][0][i] = sum over picks with left sub-key i of g_c q1_h (C' alike)
 *   grad_bn_beta = sum_t dL/dq,  grad_bn_gamma = sum_t dL/dq (acc - mean) / sqrt(var + eps)
 *   grad_W_q = (dL/dq s)^T x,    grad_x = (dL/dq s) W_q
 * Inputs are those of pkm_forward plus the forward's indices and weights and
 * grad_out [B][v] (dtype). Outputs, each fp32 and each may be NULL (not computed):
 *   grad_x        [B][d_model]        overwritten
 *   grad_W_q      [H*dq][d_model]     overwritten
 *   grad_bn_gamma [H*dq], grad_bn_beta [H*dq]  overwritten (inference BatchNorm:
 *                 the running statistics are constants and get no gradient)
 *   grad_subkeys  [H][2][n][dq/2]     overwritten
 *   grad_values   [n*n][v]            ACCUMULATED into, as in pkm_backward_values
 *   grad_scores   [B][H][k]           overwritten
 * acc is recomputed with the forward's query kernel (no BatchNorm), so the caller
 * keeps nothing from the forward beyond indices and weights. Sums over tokens are
 * in fp32 in a fixed order except sub-key rows shared by two 32-pick windows, which
 * are added atomically. Slot ids outside [0, n*n) are skipped and counted in the
 * status word. 2*B*H*k must stay below 2^31 (PKM_ERR_UNSUPPORTED otherwise: the
 * sub-key grouping sorts two contributions per pick with 32-bit positions).
 * The other gradients' chain of kernels runs on the library's helper stream (highest
 * priority) and grad_values, when requested, on `stream` beside it, joined back into
 * `stream` before the call's end.
 * workspace: at least pkm_workspace_size(s, 3) bytes, 256-byte aligned.
 */
int pkm_backward(const pkm_shape* s, const void* x, const void* W_q, const float* bn_mean,
                 const float* bn_var, const float* bn_gamma, const float* bn_beta,
                 const void* subkeys, const void* values, const int32_t* indices,
                 const float* weights, const void* grad_out, float* grad_x, float* grad_W_q,
                 float* grad_bn_gamma, float* grad_bn_beta, float* grad_subkeys,
                 float* grad_values, float* grad_scores, void* workspace, size_t workspace_bytes,
                 void* stream);

/*
 * Forward with BatchNorm in training mode ("Large Memory Layers with Product Keys",
 * Methodology: batch normalization in the query network; while the model trains, the
 * batch's own statistics normalise it, after Ioffe and Szegedy 2015):
 *   acc = x W_q^T,  mean_B = (1/B) sum_t acc[t],  var_B = (1/B) sum_t (acc[t] - mean_B)^2
 *   q = (acc - mean_B) / sqrt(var_B + eps) * gamma + beta, then as pkm_forward.
 * The running statistics move towards the batch's (PyTorch's convention):
 *   bn_running_mean <- (1 - momentum) bn_running_mean + momentum mean_B
 *   bn_running_var  <- (1 - momentum) bn_running_var  + momentum var_B B / (B - 1)
 * Arguments as pkm_forward, with bn_running_mean / bn_running_var [H*dq] fp32 updated
 * in place, momentum in [0, 1], and batch_mean / batch_var [H*dq] fp32 written: the
 * statistics that normalised the batch (biased variance), which pkm_backward_train
 * takes. B = 1 is rejected (PKM_ERR_INVALID_ARG: one token has no variance); B = 0
 * launches nothing and leaves every array as it was. Statistics are summed in fp64 in
 * chunks of 128 tokens and merged in chunk order (deterministic).
 * workspace: at least pkm_workspace_size(s, 4) bytes, 256-byte aligned.
 */
int pkm_forward_train(const pkm_shape* s, const void* x, const void* W_q,
                      float* bn_running_mean, float* bn_running_var, const float* bn_gamma,
                      const float* bn_beta, float momentum, const void* subkeys,
                      const void* values, float* out, int32_t* indices, float* weights,
                      float* scores, float* batch_mean, float* batch_var, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * pkm_backward for a forward run by pkm_forward_train: batch_mean / batch_var are the
 * statistics it wrote, and the gradient also flows through them (the backward of
 * batch normalisation):
 *   dL/dacc = gamma / sqrt(var_B + eps) (dL/dq - (1/B) sum_t dL/dq
 *                                        - xhat (1/B) sum_t dL/dq xhat),
 *   xhat = (acc - mean_B) / sqrt(var_B + eps).
 * dL/dgamma, dL/dbeta and everything else as in pkm_backward. B = 1 is rejected.
 * workspace: at least pkm_workspace_size(s, 3) bytes, 256-byte aligned.
 */
int pkm_backward_train(const pkm_shape* s, const void* x, const void* W_q,
                       const float* batch_mean, const float* batch_var, const float* bn_gamma,
                       const float* bn_beta, const void* subkeys, const void* values,
                       const int32_t* indices, const float* weights, const void* grad_out,
                       float* grad_x, float* grad_W_q, float* grad_bn_gamma, float* grad_bn_beta,
                       float* grad_subkeys, float* grad_values, float* grad_scores,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * pkm_backward_values without a workspace. The pages have no counterpart: this is
 * a convenience of this library. It is for callers that cannot allocate device
 * memory where they run the backward (a runtime that hands out all device memory
 * from its own pool and forbids other allocations while it executes, or a plugin
 * host that passes device pointers but no allocator). Arguments and results are
 * those of pkm_backward_values; the caller still passes inputs and outputs.
 *
 * Scratch: one fixed device array of about 44.2 MiB inside libpkm.so, held on every
 * GPU that loads the library until the process exits. Limits: n*n <= 1,048,576 slots,
 * B*H*k <= 2,097,152 picks and v <= 2048; larger shapes return PKM_ERR_UNSUPPORTED
 * before any launch. The call allocates nothing (no cudaMalloc, no library allocator).
 * The first call on a device looks up the array's device address with that device
 * current; make that first call before any stream capture. All calls share the
 * one array (each call clears what must start at zero), so calls that overlap on
 * the GPU -- on different streams, or from different threads -- race and must
 * not be issued. Slot ids outside [0, n*n) are skipped as in pkm_backward_values,
 * but the status word is not readable through pkm_device_status.
 */
int pkm_backward_values_noalloc(const pkm_shape* s, const void* values, const int32_t* indices,
                                const float* weights, const void* grad_out, float* grad_values,
                                float* grad_scores, void* stream);

/*
 * Memory utilisation of one batch ("Large Memory Layers with Product Keys", gptget.net
 * summary, Key Results: BatchNorm in the query network raises the share of memory
 * slots in use above 80 %): the number of distinct slots among the B*H*k picks.
 *   indices  [B][H][k] int32, as written by pkm_forward
 *   hits     one device uint64, overwritten with the count
 * Only B, H, n and k of the shape are read. Ids outside [0, n*n) are not counted and
 * set the status word (PKM_ERR_DEVICE).
 * workspace: at least pkm_workspace_size(s, 2) bytes (status word + one bit per slot).
 */
int pkm_slot_usage(const pkm_shape* s, const int32_t* indices, unsigned long long* hits,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---------------------------------------------------------------------------
 * The transformer block around the layer ("Large Memory Layers with Product Keys":
 * the memory takes the place of a feed-forward sub-layer of a transformer and is
 * trained end-to-end with it): layer norm before a sub-layer, the dense sub-layers,
 * and the optimizer step. Conventions as above (caller-owned contiguous device
 * arrays, 16-byte aligned; asynchronous on `stream`; the device that owns the arrays
 * is current; arguments validated before any launch). Arrays that are written (the workspace
 * too) overlap no other array that the call reads or writes but where an entry says that
 * two may be the same array (the norm and the dense layer refuse it:
 * PKM_ERR_INVALID_ARG). Calls take no lock that
 * outlives them and share no scratch, so calls on different streams may overlap if
 * their workspaces and outputs differ.
 * ---------------------------------------------------------------------------
 */

/* Layer norm sizes and types; every *_dtype is a pkm_dtype. */
typedef struct {
  int64_t rows;       /* rows (tokens), < 2^31; 0 is allowed, and then the per-row pointers may be
                         NULL */
  int32_t d;          /* row length, 1 <= d <= 16384 (PKM_ERR_UNSUPPORTED above) */
  int32_t x_dtype;    /* x and sum */
  int32_t add_dtype;  /* add; in the backward grad_sum */
  int32_t y_dtype;    /* y; in the backward grad_y */
  int32_t grad_dtype; /* grad_x (backward only) */
  float eps;          /* added to the variance */
} pkm_norm_shape;

/*
 * Layer norm, with the residual stream's addition before it:
 *   h = x + add (added in fp32, rounded to x's type; h = x when add is NULL)
 *   mean = (1/d) sum_j h_j,  rstd = 1 / sqrt((1/d) sum_j (h_j - mean)^2 + eps)
 *   y_j = (h_j - mean) rstd gamma_j + beta_j
 *   x      [rows][d]  x_dtype         add   [rows][d]  add_dtype, may be NULL
 *   gamma, beta  [d]  fp32            (beta may be NULL: no bias)
 * Outputs (overwritten):
 *   y      [rows][d]  y_dtype
 *   sum    [rows][d]  x_dtype         h; required with add, must be NULL without
 *   mean, rstd  [rows] fp32           each may be NULL
 * sum or y may be the same array as x or add where the types are equal (in place).
 * Statistics are computed in fp32 from the row held
 * on chip, the variance from the centred values.
 */
int pkm_layernorm_forward(const pkm_norm_shape* s, const void* x, const void* add,
                          const float* gamma, const float* beta, void* y, void* sum, float* mean,
                          float* rstd, void* stream);

/* Bytes of workspace pkm_layernorm_backward needs; 0 if the shape is invalid. Only rows
 * and d are read. A workspace for some rows serves fewer as well. */
size_t pkm_norm_workspace_size(const pkm_norm_shape* s);

/*
 * Backward of pkm_layernorm_forward. x is the normalised array (sum where there was an
 * add), mean and rstd are the forward's. With xhat = (x - mean) rstd, t = grad_y gamma:
 *   grad_x = rstd (t - (1/d) sum_j t_j - xhat (1/d) sum_j t_j xhat_j) + grad_sum
 *   grad_gamma = sum_rows grad_y xhat,   grad_beta = sum_rows grad_y
 *   grad_y [rows][d] y_dtype, x [rows][d] x_dtype, mean, rstd [rows] and gamma [d] fp32
 *   grad_sum [rows][d] add_dtype: gradient that reaches the residual stream past the
 *            norm; may be NULL
 *   grad_x [rows][d] grad_dtype: overwritten. It is the gradient of x and of add alike.
 *            It may be the same array as grad_y, grad_sum or x where the types are equal.
 *   grad_gamma, grad_beta [d] fp32: overwritten (zero when rows is 0); each may be NULL
 * Column sums are in fp32 in a fixed order: the result is bit-for-bit the same on every
 * run. workspace: pkm_norm_workspace_size(s) bytes, 256-byte aligned.
 */
int pkm_layernorm_backward(const pkm_norm_shape* s, const void* grad_y, const void* x,
                           const float* mean, const float* rstd, const float* gamma,
                           const void* grad_sum, void* grad_x, float* grad_gamma,
                           float* grad_beta, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Activations of the dense layer: relu; gelu(v) = v Phi(v) with the normal distribution
 * Phi (not its tanh approximation); silu(v) = v / (1 + exp(-v)). fp32 results of gelu and silu,
 * and each term of their slopes, are within 2^-19 of themselves while Phi or exp(v) is above
 * 2^-126 (0 below); bf16 results within 2^-15 before they are rounded. */
enum { PKM_ACT_NONE = 0, PKM_ACT_RELU = 1, PKM_ACT_GELU = 2, PKM_ACT_SILU = 3 };

/* Dense layer sizes and types. */
typedef struct {
  int64_t M;           /* rows (tokens), up to 2^31 - 257; 0 is allowed, and then the per-row
                          pointers may be NULL */
  int32_t N;           /* output width, 1 <= N <= 2^20 */
  int32_t K;           /* input width, 1 <= K <= 2^20 */
  int32_t dtype;       /* pkm_dtype of x, W, pre and, in the backward, grad_y */
  int32_t out_dtype;   /* pkm_dtype of y and residual; in the backward of grad_x */
  int32_t activation;
} pkm_linear_shape;

/* Bytes of workspace of pkm_linear_forward (for_backward = 0) or pkm_linear_backward (1);
 * 0 if the shape is invalid or not supported. Fewer rows may need more (their products are
 * cut into parts): a workspace for several M holds the largest of their sizes. */
size_t pkm_linear_workspace_size(const pkm_linear_shape* s, int for_backward);

/*
 * Dense layer: pre = x W^T + bias,  y = activation(pre) + residual.
 *   x [M][K], W [N][K]  dtype;  bias [N] fp32, may be NULL;  residual [M][N] out_dtype, may be
 *   NULL (or the same array as y: in place)
 * Outputs (overwritten): y [M][N] out_dtype;  pre [M][N] dtype, may be NULL: what
 * pkm_linear_backward takes.
 * Products accumulate in fp32 on the tensor cores, which may cut 2^-24 of a running sum every 16
 * terms; sums start anew every 256 terms and are added to nearest where the result is fp32, or
 * has more than 2^15 terms. fp32 operands are split into three bf16 planes whose sum is the
 * value to 2^-24, and the products above 2^-24 of the largest are added; so an infinite
 * operand makes its sums infinite or NaN, and below 2^-100 an operand is its planes to
 * 2^-134, not relatively. Small fp32 layers multiply in fp32 on the CUDA cores instead, with
 * a sum of its own for every 32 terms. y is computed from pre before pre is rounded. Few rows
 * (up to 8, in bf16 16 or 32) take kernels that stream W once. M N and M K are below 2^38.
 * workspace: pkm_linear_workspace_size(s, 0) bytes, 256-byte aligned; its status word
 * (pkm_device_status) records a bounded wait that ran out. A call without work (M = 0, or in the
 * backward no gradient asked for) launches no kernel and leaves the status word as it was.
 */
int pkm_linear_forward(const pkm_linear_shape* s, const void* x, const void* W, const float* bias,
                       const void* residual, void* y, void* pre, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * Backward of pkm_linear_forward. With d = grad_y activation'(pre) (relu'(0) = 0):
 *   grad_x [M][K] out_dtype = d W,  grad_W [N][K] fp32 = d^T x,  grad_bias [N] fp32 = sum_rows d
 * each overwritten and each may be NULL (not computed). The residual's gradient is grad_y.
 *   x, W as in the forward; grad_y [M][N] dtype; pre [M][N] dtype as the forward wrote it
 *   (not read, may be NULL, without an activation)
 * d is an fp32 value. With an activation and in fp32 layers (but small ones) it enters the
 * products as three bf16 planes whose sum is d to 2^-24; in a bf16 layer's bf16 grad_x as two,
 * d to 2^-16 (relu: d is bf16 itself). Column sums add in a fixed order; all results are
 * bit-for-bit the same on every run.
 * workspace: pkm_linear_workspace_size(s, 1) bytes, 256-byte aligned, status word as above.
 */
int pkm_linear_backward(const pkm_linear_shape* s, const void* x, const void* W,
                        const void* grad_y, const void* pre, void* grad_x, float* grad_W,
                        float* grad_bias, void* workspace, size_t workspace_bytes, void* stream);

/* One tensor of an AdamW step. */
typedef struct {
  void* param;          /* [n] param_dtype, updated */
  void* grad;           /* [n] grad_dtype; set to zero after it was read with zero_grad */
  float* master;        /* [n] fp32 copy that carries the parameter: updated, and param becomes
                           its rounding. NULL: param carries itself */
  void* m;              /* first moment: [n] fp32, or e4m3 codes with state_bits 8 */
  void* v;              /* second moment: [n] fp32, or e4m3 codes of its square root with
                           state_bits 8 */
  float* m_scale;       /* state_bits 8: [ceil(n / 256)] the scale of each 256 elements' codes */
  float* v_scale;       /* (NULL with state_bits 32) */
  int64_t n;            /* elements, 0 <= n < 2^38 */
  int32_t param_dtype;  /* pkm_dtype */
  int32_t grad_dtype;   /* pkm_dtype */
  int32_t state_bits;   /* 32 or 8 */
  float weight_decay;   /* >= 0 */
  float lr_scale;       /* the tensor's learning rate over the call's, >= 0 */
} pkm_adamw_tensor;

typedef struct {
  double lr;            /* >= 0 */
  double beta1, beta2;  /* in [0, 1) */
  double eps;           /* > 0 */
  double grad_scale;    /* gradients are multiplied by it (clipping, loss scaling) */
  int64_t step;         /* t, 1 for the first step */
  uint32_t seed;        /* of the dither of 8-bit states */
  int32_t zero_grad;    /* 1: gradients are cleared for the next step (pkm_backward
                           accumulates into grad_values) */
} pkm_adamw_hyper;

/*
 * One AdamW step (Loshchilov and Hutter, decoupled weight decay) over a list of tensors:
 *   g = grad grad_scale,  m <- beta1 m + (1 - beta1) g,  v <- beta2 v + (1 - beta2) g^2
 *   p <- p (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32, with lr = hyper.lr lr_scale (quotients, and square roots of fp32 states, to 2^-22;
 * second moments of 8-bit states that are below 2^-110 to fewer bits). The moments that move p are
 * the new ones before they are rounded to 8 bits.
 * 8-bit states (after the block-wise states of Dettmers et al., "8-bit Optimizers via
 * Block-wise Quantization"): m and r = sqrt(v) as fp8 e4m3 codes, each block of 256
 * elements (counted from the tensor's start) with its scale s = the smallest power of two,
 * at least 2^-100, with |value| <= 448 s all over the block (NaN where a value is not
 * finite: such a block's states are NaN from then on). A value is code * s. A power of two
 * keeps the codes' grid where it is from one step to the next. m / s is rounded to nearest
 * even. One step moves r by a small part of a code, which rounding to nearest would drop
 * every time: q = r / s is rounded after a dither, to the code nearest to q + u ulp, with
 * ulp the code spacing at q and u = (b - 32767.5) / 65536, b the 16 low (even elements) or
 * high (odd elements) bits of mix(i / 2 xor key), key = mix(mix(seed + 0x9e3779b9 t) xor
 * 0x9e3779b9 index), index the tensor's place in the list, mix MurmurHash3's 32-bit
 * finaliser, all modulo 2^32. (Codes below a power of two lie half as far apart, so a q
 * within ulp / 4 above one may go to the code below it, half an ulp down.) What is above 0
 * stays at least the smallest code, 2^-9. All zeros (codes and scales) are the initial states.
 *   dyn: NULL, or three device fp32 {lr, t, grad_scale} read when the step runs, in the
 *        place of hyper's (t a whole number >= 1): a captured step takes new values at
 *        every replay.
 * An array may not appear twice in the list. Tensors with n = 0 are skipped (their index
 * counts). Arrays behind the list may be freed when the call returns (the list is copied
 * into the launches).
 */
int pkm_adamw_step(const pkm_adamw_tensor* tensors, int64_t count, const pkm_adamw_hyper* hyper,
                   const float* dyn, void* stream);

/*
 * Synchronises `stream`, reads the status word that the kernels of the last call
 * on this workspace wrote (each call clears it when it starts), clears it and
 * returns PKM_OK, PKM_ERR_DEVICE or PKM_ERR_CUDA. This is the only entry point
 * that blocks the host.
 */
int pkm_device_status(void* workspace, void* stream);

/*
 * Stage timing (a measurement aid; the pages have no counterpart). While enabled,
 * every kernel a call launches is bracketed by two CUDA events recorded on the stream
 * it runs on, and so is the whole call (on `stream`). Forward stages: 0 query network,
 * 1 per-half scores and best 32, 2 candidate top-k + softmax + value gather, 3 the
 * whole call. Backward stages: 0 grad wrt kept scores, 1 slot grouping and row sums,
 * 3 the whole call. The events are owned by the library (host-side handles only).
 * pkm_trace_read waits for the recorded events of `pass` (0 forward, 1 backward),
 * writes the summed milliseconds per stage into stage_ms[0..max_stages) (a stage that
 * runs several launches per call, or overlaps another stage, sums their own
 * durations), the number of traced calls into *calls, and the number of kernels the
 * library launched since the last read (all passes, traced or not) into *launches;
 * then forgets them. Returns PKM_OK, PKM_ERR_INVALID_ARG or PKM_ERR_CUDA.
 */
int pkm_trace_enable(int on);
int pkm_trace_read(int pass, double* stage_ms, int max_stages, int64_t* calls,
                   int64_t* launches);

/*
 * Implementation switches (a convenience of this library; the pages have no
 * counterpart). Process-wide, for every device; a change applies to calls made after
 * it. The environment variables PKM_PATH (auto | tc | simt | small_fused | small_split) and
 * PKM_SUBBATCHES (1..4)
 * give the initial values and are read once, at the first call that needs them.
 *   PKM_OPT_PATH        PKM_PATH_AUTO (default): the small-batch kernels for small
 *                       batches (see pkm_forward), else the tensor-core kernels where
 *                       the layer fits
 *                       their tiles (bf16, d_model and dq/2 multiples of 64, n a
 *                       multiple of 256, H*dq <= 4096), else the CUDA-core kernels;
 *                       PKM_PATH_TC: never the small-batch kernels;
 *                       PKM_PATH_SIMT: always the CUDA-core kernels;
 *                       PKM_PATH_SMALL_FUSED: the small-batch path for every batch
 *                       it supports (up to 512 tokens), as the one cooperative
 *                       kernel;
 *                       PKM_PATH_SMALL_SPLIT: the same, as the three kernels.
 *   PKM_OPT_SUBBATCHES  1 (default) to 4: sub-batches of the pipelined tensor-core
 *                       forward (see pkm_forward). The forward's workspace size
 *                       depends on it: query it after setting the option.
 * pkm_set_option returns PKM_OK or PKM_ERR_INVALID_ARG (unknown option or value);
 * pkm_get_option returns the current value or PKM_ERR_INVALID_ARG.
 */
enum { PKM_OPT_PATH = 0, PKM_OPT_SUBBATCHES = 1 };
enum {
  PKM_PATH_AUTO = 0,
  PKM_PATH_TC = 1,
  PKM_PATH_SIMT = 2,
  PKM_PATH_SMALL_FUSED = 3,
  PKM_PATH_SMALL_SPLIT = 4
};
int pkm_set_option(int option, int value);
int pkm_get_option(int option);

/* Static string for a status code. */
const char* pkm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* PKM_H_ */
